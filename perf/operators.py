"""The operators of a preference or policy fine-tuning step as measured cases.

Four operators around the adapted linear: the log-probabilities of the labels
under a head's logits (``score``), the preference loss of chosen and rejected
sequences with its gradient in the logits (``preference``), the clipped policy
loss with a KL term and its gradient in the logits (``policy``), and the
optimiser step that orthogonalises an adapter factor's update (``muon``).
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
NS = (3.4445, -4.7750, 2.0315)  # coefficients of one Newton-Schulz step
LARGEST = 1 << 29               # logits of the largest listed case


def listed():
    return [
        # scoring one short answer of 24 tokens against a 32000-word head: latency
        dict(name="score_short", op="score", T=24, V=32000, pad=0, dtype="bf16", masked=0.0, tau=1.0),
        # scoring a batch under fp32 logits; an odd vocabulary inside a head padded to whole tiles
        dict(name="score_odd_f32", op="score", T=4093, V=50021, pad=27, dtype="f32", masked=0.1, tau=1.0),
        # one preference pair of a few words, fp32 logits of a small vocabulary: the smallest training call
        dict(name="pref_one_pair", op="preference", T=61, V=8191, pad=1, dtype="f32", masked=0.3, tau=1.0, P=1,
             cut=3, kind="sigmoid", average=False, smooth=0.0),
        # an ordinary preference batch: 8 pairs, 4096 tokens, the prompts masked
        dict(name="pref_batch", op="preference", T=4096, V=32000, pad=0, dtype="bf16", masked=0.4, tau=1.0, P=8,
             cut=5, kind="sigmoid", average=False, smooth=0.1),
        # a large vocabulary, length-normalised squared loss, few tokens masked
        dict(name="pref_large_vocab", op="preference", T=4096, V=131072, pad=0, dtype="bf16", masked=0.1, tau=1.0,
             P=16, cut=7, kind="squared", average=True, smooth=0.0),
        # the policy loss of a few sampled tokens, fp32 logits, sampled at a temperature of 0.8
        dict(name="policy_few_f32", op="policy", T=96, V=32000, pad=0, dtype="f32", masked=0.1, tau=1.25, kl=0.05),
        # an ordinary batch of 4096 sampled tokens
        dict(name="policy_batch", op="policy", T=4096, V=32000, pad=0, dtype="bf16", masked=0.2, tau=1.0, kl=0.05),
        # a large vocabulary of an odd size in a padded head
        dict(name="policy_large_vocab", op="policy", T=4096, V=131071, pad=1, dtype="bf16", masked=0.1, tau=1.0,
             kl=0.0),
        # one rank-8 factor of a 256 x 256 layer: latency
        dict(name="muon_small", op="muon", n=1, rows=8, cols=256, nesterov=True),
        # the B factors of three sections with an odd rank and an odd height
        dict(name="muon_odd", op="muon", n=3, rows=1001, cols=7, nesterov=False),
        # the B factors of one projection in every layer of a 32-layer stack at r = 16
        dict(name="muon_stack_b", op="muon", n=32, rows=11008, cols=16, nesterov=True),
        # the A factors of one projection in every layer of an 80-layer stack at r = 64
        dict(name="muon_stack_a", op="muon", n=80, rows=64, cols=8192, nesterov=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["score", "preference", "policy", "muon"])
    if op == "muon":
        short, long = rng.randint(1, 64), _spread(rng, 64, 22016)
        n = _spread(rng, 1, max(1, min(80, (80 * 64 * 8192) // (64 * long))))
        rows, cols = (short, long) if rng.random() < 0.5 else (long, short)
        return dict(op=op, n=n, rows=rows, cols=cols, nesterov=rng.random() < 0.7)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = _spread(rng, 200, 131072)
    most = LARGEST * 2 // SIZE[dtype]
    T = _spread(rng, 4, min(16384, most // (V + 64)))
    case = dict(op=op, T=T, V=V, pad=rng.choice([0, 0, 1, 5, (-V) % 64]), dtype=dtype,
                masked=rng.choice([0.0, 0.1, 0.4, 0.7]), tau=rng.choice([1.0, 1.0, 0.5, 1.25]))
    if op == "preference":
        case.update(P=rng.randint(1, max(1, min(16, T // 4))), cut=rng.randint(0, 10**6),
                    kind=rng.choice(["sigmoid", "hinge", "squared"]), average=rng.random() < 0.5,
                    smooth=rng.choice([0.0, 0.1]))
        if case["kind"] != "sigmoid":
            case["smooth"] = 0.0
    if op == "policy":
        case.update(kl=rng.choice([0.0, 0.02, 0.1]))
    return case


def _offsets(case):
    """Offsets of the 2P sequences of a case: ragged, an empty one now and then."""
    rng = random.Random(case["cut"])
    cuts = sorted(rng.randint(0, case["T"]) for _ in range(2 * case["P"] - 1))
    return [0] + cuts + [case["T"]]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * seed + 17)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    if case["op"] == "muon":
        n, rows, cols = case["n"], case["rows"], case["cols"]
        few = min(4, rows, cols)

        def update():  # a few strong directions over noise, as an adapter's gradients have
            return 1e-3 * (torch.bmm(normal(n, rows, few), normal(n, few, cols)) + 0.5 * normal(n, rows, cols))

        W = normal(n, rows, cols) * (cols ** -0.5 if rows <= cols else 0.01)
        return dict(case=case, G=update().bfloat16(), m=4 * update(), W=W, P=W.bfloat16())

    T, V = case["T"], case["V"]
    logits = torch.empty(T, V + case["pad"], device=DEV, dtype=DTYPES[case["dtype"]])
    for at in range(0, T, 1024):
        logits[at:at + 1024] = normal(min(1024, T - at), V + case["pad"]) * 2
    logits = logits[:, :V]
    labels = torch.randint(0, V, (T,), device=DEV, generator=g)
    rows = torch.arange(T, device=DEV)
    # most labels are likely ones
    logits[rows, labels] += (torch.rand(T, device=DEV, generator=g) * 14).to(logits.dtype)
    labels[torch.rand(T, device=DEV, generator=g) < case["masked"]] = -100
    state = dict(case=case, logits=logits, labels=labels.int())
    if case["op"] == "score":
        return state
    logp = torch.cat([torch.log_softmax(logits[at:at + 1024].float() * case["tau"], 1) for at in range(0, T, 1024)] if
                     T * V < 1 << 26 else
                     [torch.log_softmax(logits[at:at + 1024].float() * case["tau"], 1).gather(
                         1, labels[at:at + 1024, None].clamp(min=0).long()) for at in range(0, T, 1024)])
    logp = (logp.gather(1, labels[:, None].clamp(min=0).long()) if logp.shape[1] == V else logp)[:, 0]
    # the reference differs a little at each token, and the policy has gained on it as a whole
    state["ref_logp"] = torch.where(labels >= 0, logp - 0.1 + 0.2 * normal(T), 0.0)
    if case["op"] == "preference":
        P = case["P"]
        state["cu"] = torch.tensor(_offsets(case), device=DEV, dtype=torch.int32)
        state["weight"] = torch.full((P,), 1.0 / P, device=DEV)
        return state
    # sampled some steps ago: ratios around one, none within rounding of where the clipping begins
    off = 0.15 * normal(T)
    for edge in (math.log(0.8), math.log(1.2)):
        off = torch.where((off - edge).abs() < 2e-3, off + 0.01, off)
    state["old_logp"] = torch.where(labels >= 0, logp - off, 0.0)
    state["advantages"] = normal(T)
    state["weight"] = torch.full((T,), 1.0 / T, device=DEV)
    return state


# ------------------------------------------------------------ plain forms --

def _stats(logits, labels, tau):
    """t = tau (z - max z), ln sum exp t, the label's log-probability, and which tokens count.  The sum over the
    vocabulary is taken in 64 bits: its error is the same for every token of a kind and adds up in a sequence's sum."""
    z = logits.float()
    t = (z - z.max(dim=1, keepdim=True).values) * tau
    log_sum = t.exp().sum(dim=1, keepdim=True, dtype=torch.float64).log()
    counted = (labels >= 0) & (labels < logits.shape[1])
    index = torch.where(counted, labels, 0).long()[:, None]
    logp = (t.gather(1, index) - log_sum)[:, 0].float()
    return t, log_sum.float(), torch.where(counted, logp, 0.0), counted, index


def _grad(t, log_sum, index, g, tau, dtype):
    d = (t - log_sum).exp().neg()
    d.scatter_add_(1, index, torch.ones_like(index, dtype=d.dtype))
    return (d * (g * tau)[:, None]).to(dtype)


def _plain_preference(s):
    c, cu, labels = s["case"], s["cu"].long(), s["labels"]
    t, log_sum, logp, counted, index = _stats(s["logits"], labels, c["tau"])
    T, P, beta = c["T"], c["P"], 0.1

    def sums(v):  # over each sequence, in 64 bits: thousands of terms whose small differences count
        total = torch.cat([v.new_zeros(1, dtype=torch.float64), v.double().cumsum(0)])
        return total[cu[1:]] - total[cu[:-1]]

    number = sums(counted) if c["average"] else torch.ones(2 * P, device=DEV, dtype=torch.float64)
    gain = sums(torch.where(counted, logp.double() - s["ref_logp"].double(), 0.0)) / number.clamp(min=1)
    diff = gain[:P] - gain[P:]
    h = beta * diff
    if c["kind"] == "sigmoid":
        e = c["smooth"]
        low = torch.log1p((-h.abs()).exp())
        loss = (1 - e) * (low + (-h).clamp(min=0)) + e * (low + h.clamp(min=0))
        dh = -(1 - e) / (1 + h.exp()) + e / (1 + (-h).exp())
    elif c["kind"] == "hinge":
        loss, dh = (1 - h).clamp(min=0), torch.where(h < 1, -1.0, 0.0).double()
    else:
        loss, dh = (diff - 1 / (2 * beta)).square(), 2 * (diff - 1 / (2 * beta)) / beta
    per_seq = torch.cat([dh, -dh]) * beta * s["weight"].double().repeat(2) / number.clamp(min=1)
    which = torch.searchsorted(cu[1:], torch.arange(T, device=DEV), right=True)
    dlogp = torch.where(counted, per_seq[which], 0.0).float()
    return (loss.float(), (beta * gain).float(), logp,
            _grad(t, log_sum, index, dlogp, c["tau"], s["logits"].dtype))


def _plain_policy(s):
    c = s["case"]
    t, log_sum, logp, counted, index = _stats(s["logits"], s["labels"], c["tau"])
    A = s["advantages"]
    ratio = (logp - s["old_logp"]).exp()
    clipped = ratio.clamp(0.8, 1.2)
    loss = -torch.minimum(ratio * A, clipped * A)
    inside = torch.where(A >= 0, ratio <= 1.2, ratio >= 0.8)
    g = torch.where(inside, -ratio * A, 0.0)
    d = s["ref_logp"] - logp
    kl = torch.expm1(d) - d
    loss = loss + c["kl"] * kl
    g = g - c["kl"] * torch.expm1(d)
    g = torch.where(counted, g * s["weight"], 0.0)
    return (torch.where(counted, loss, 0.0), torch.where(counted, kl, 0.0), logp,
            _grad(t, log_sum, index, g, c["tau"], s["logits"].dtype))


def _plain_muon(s):
    c, G, m, W = s["case"], s["G"].float(), s["m"], s["W"]
    m.mul_(0.95).add_(G)
    X = G + 0.95 * m if c["nesterov"] else m
    tall = c["rows"] > c["cols"]
    if tall:
        X = X.transpose(1, 2).contiguous()
    X = X / (X.square().sum(dim=(1, 2), keepdim=True).sqrt() + 1e-7)
    a, b, cc = NS
    for _ in range(5):
        gram = torch.bmm(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.bmm(b * gram + cc * torch.bmm(gram, gram), X)
    if tall:
        X = X.transpose(1, 2)
    W.mul_(1 - 2e-3 * 0.01).sub_(X, alpha=2e-3 * max(1.0, c["rows"] / c["cols"]) ** 0.5)
    s["P"].copy_(W)
    return W, m, s["P"]


def run(state):
    c, op = state["case"], state["case"]["op"]
    if not own:
        if op == "score":
            return _stats(state["logits"], state["labels"], c["tau"])[2]
        return {"preference": _plain_preference, "policy": _plain_policy, "muon": _plain_muon}[op](state)
    import parameter_efficient_fine_nf4_amd as q
    if op == "score":
        return q.token_logprobs(state["logits"], state["labels"], inv_temperature=c["tau"])
    if op == "preference":
        logits, labels = state["logits"], state["labels"]
        logp, stats = q.token_logprobs(logits, labels, inv_temperature=c["tau"], save_stats=True)
        loss, reward, dlogp = q.preference_loss(logp, labels, c["V"], state["cu"], beta=0.1,
                                                ref_logp=state["ref_logp"], kind=c["kind"], average=c["average"],
                                                label_smoothing=c["smooth"], weight=state["weight"])
        dlogits = q.token_logprobs_backward(dlogp, logits, labels, stats, inv_temperature=c["tau"])
        return loss, reward, logp, dlogits
    if op == "policy":
        return q.policy_loss(state["logits"], state["labels"], state["advantages"], old_logp=state["old_logp"],
                             ref_logp=state["ref_logp"], weight=state["weight"], clip_low=0.2, clip_high=0.2,
                             kl_coef=c["kl"], inv_temperature=c["tau"])
    q.muon_step(state["P"], state["W"], state["G"], state["m"], lr=2e-3, momentum=0.95, nesterov=c["nesterov"],
                weight_decay=0.01)
    return state["W"], state["m"], state["P"]


def work(case):
    if case["op"] == "muon":
        count = case["n"] * case["rows"] * case["cols"]
        short = min(case["rows"], case["cols"])
        return {"bytes": 20 * count, "flops": 4 * short * count + 34 * case["n"] * short ** 3}
    T, V, size = case["T"], case["V"], SIZE[case["dtype"]]
    read = (1 - case["masked"]) * T * V * size  # a masked token's logits take part in nothing
    if case["op"] == "score":
        return {"bytes": read + 8 * T, "flops": 4 * T * V}
    return {"bytes": read + T * V * size + 28 * T, "flops": 8 * T * V}


# ---------------------------------------------------------- in 64 bits -----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "muon":
        G, m, W = s["G"].double(), s["m"].double(), s["W"].double()
        m = 0.95 * m + G
        u = G + 0.95 * m if case["nesterov"] else m
        for i in range(case["n"]):
            x = u[i] if case["rows"] <= case["cols"] else u[i].t().contiguous()
            x = x / (torch.linalg.vector_norm(x) + 1e-7)
            eye = torch.eye(x.shape[0], dtype=torch.float64, device=DEV)
            for _ in range(5):
                sq = x @ x.t().contiguous()
                x = (NS[0] * eye + NS[1] * sq + NS[2] * (sq @ sq)) @ x
            step = x if case["rows"] <= case["cols"] else x.t()
            W[i] = W[i] * (1 - 2e-3 * 0.01) - 2e-3 * math.sqrt(max(1.0, case["rows"] / case["cols"])) * step
        return W, m, W
    logits, labels, T, V, tau = s["logits"], s["labels"].tolist(), case["T"], case["V"], case["tau"]
    step = max(1, (1 << 26) // V)
    logp = torch.zeros(T, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, dtype=torch.float64, device=DEV)
    known = torch.tensor([y >= 0 for y in labels], device=DEV)
    at_label = torch.tensor([max(y, 0) for y in labels], device=DEV)
    for i in range(0, T, step):
        z = logits[i:i + step].double() * tau
        lse[i:i + step] = torch.logsumexp(z, 1)
        logp[i:i + step] = z[torch.arange(z.shape[0], device=DEV), at_label[i:i + step]] - lse[i:i + step]
    logp[~known] = 0
    if case["op"] == "score":
        return logp
    ref = s["ref_logp"].double()
    g = torch.zeros(T, dtype=torch.float64, device=DEV)
    if case["op"] == "preference":
        P, beta, cu = case["P"], 0.1, _offsets(case)
        gains, counts = [], []
        for k in range(2 * P):
            part = slice(cu[k], cu[k + 1])
            counts.append(max(1, int(known[part].sum())) if case["average"] else 1)
            gains.append(float(((logp - ref) * known)[part].sum()) / counts[-1])
        losses = []
        for p in range(P):
            d = gains[p] - gains[P + p]
            h, e = beta * d, case["smooth"]
            if case["kind"] == "sigmoid":
                up = 1 / (1 + math.exp(-h))
                losses.append(-(1 - e) * math.log(up) - e * math.log(1 - up))
                slope = beta * (e - (1 - up))  # d/dh: -(1-e)(1-up) + e up = up - 1 + e
            elif case["kind"] == "hinge":
                losses.append(max(0.0, 1 - h))
                slope = -beta if h < 1 else 0.0
            else:
                losses.append((d - 0.5 / beta) ** 2)
                slope = 2 * (d - 0.5 / beta)
            for k, sign in ((p, 1), (P + p, -1)):
                g[cu[k]:cu[k + 1]] = sign * slope * float(s["weight"][p]) / counts[k]
        head = [torch.tensor(losses, device=DEV, dtype=torch.float64),
                beta * torch.tensor(gains, device=DEV, dtype=torch.float64), logp]
    else:
        A, r = s["advantages"].double(), torch.exp(logp - s["old_logp"].double())
        first, second = r * A, r.clamp(0.8, 1.2) * A
        d = ref - logp
        kl = torch.exp(d) - d - 1
        g = -torch.where(first <= second, first, 0.0) + case["kl"] * (1 - torch.exp(d))
        g = g * s["weight"].double()
        head = [torch.where(known, -torch.minimum(first, second) + case["kl"] * kl, 0.0),
                torch.where(known, kl, 0.0), logp]
    g = torch.where(known, g, 0.0) * tau
    grad = torch.empty(T, V, dtype=torch.float64, device=DEV)
    for i in range(0, T, step):
        z = logits[i:i + step].double() * tau
        part = -torch.exp(z - lse[i:i + step, None])
        part[torch.arange(z.shape[0], device=DEV), at_label[i:i + step]] += 1
        grad[i:i + step] = part * g[i:i + step, None]
    return (*head, grad)
