"""The vocabulary-loss operators: cases, inputs, plain forms and 64-bit values.

A language model's last product, logits = x . w^T (x [T,H] hidden states, w the
vocabulary's weights), exists only to be reduced: to a softmax cross entropy
against one target per row, or to a divergence from a teacher's top-k logits.
Four operators:

  xent      forward   loss_t = lse_t - z_t[y_t] (+ zeta lse_t^2), lse_t = log sum_v exp z_t[v]
  xent      backward  dz_t = g_t ((1 + 2 zeta lse_t) p_t - onehot(y_t)), dx = dz . w, dw = dz^T . x
  distill   forward   q_t = softmax(teacher_t / tau) over the row's K entries,
                      loss_t = tau^2 sum_k q_tk (log q_tk - z_t[i_tk] / tau + lse_t), lse_t = log sum_v exp(z_t[v] / tau)
  distill   backward  dz_t = g_t tau (p_t - q_t), p_t = exp(z_t / tau - lse_t), dx and dw as above

Rows whose target is -100 (xent), or whose entries are all -1 (distill), have
loss 0 and no gradient; single entries of -1 are padding.

Where `own` is false `run` computes them with elementary torch operations in
fp32; where it is true it calls dense_gemm_work_amd.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    def c(name, op, T, V, H, dtype="bf16", layout="nk", **kw):
        return dict({"name": name, "op": op, "T": T, "V": V, "H": H, "dtype": dtype, "layout": layout, "zeta": 0.0,
                     "K": 0, "tau": 1.0}, **kw)

    return [
        # the log probability of one token after one decoding step: latency
        c("xent fwd 1 token", "xent_fwd", 1, 8192, 1536),
        # scoring one token of each request of a decode batch, vocabulary of an odd size: the weights' stream
        c("xent fwd 96 tokens", "xent_fwd", 96, 50001, 2048, "fp16"),
        # evaluating a document: perplexity over long context
        c("xent fwd 4096 tokens", "xent_fwd", 4096, 131072, 4096),
        # fine-tuning on one short answer, weights stored [H,V]
        c("xent bwd 64 tokens", "xent_bwd", 64, 32000, 2048, layout="kn"),
        # a ragged micro-batch of a small model trained in fp16
        c("xent bwd 777 tokens", "xent_bwd", 777, 50001, 1536, "fp16", zeta=1e-4),
        # an ordinary training micro-batch
        c("xent bwd 2048 tokens", "xent_bwd", 2048, 32768, 2048),
        # the largest: a long micro-batch over a large vocabulary, with the z term
        c("xent bwd 8192 tokens", "xent_bwd", 8192, 131072, 4096, zeta=1e-4),
        # on-policy distillation scores single tokens
        c("distill fwd 2 tokens", "distill_fwd", 2, 32768, 2048, K=20, tau=2.0),
        # validation of a distilled model
        c("distill fwd 2048 tokens", "distill_fwd", 2048, 65536, 4096, K=64, tau=1.0),
        # a ragged batch against few teacher entries
        c("distill bwd 333 tokens", "distill_bwd", 333, 50001, 2048, "fp16", K=8, tau=2.0),
        # weights stored [H,V], many entries
        c("distill bwd 1024 tokens", "distill_bwd", 1024, 32768, 1536, layout="kn", K=128, tau=1.5),
        # distillation of a long micro-batch
        c("distill bwd 4096 tokens", "distill_bwd", 4096, 65536, 4096, K=64, tau=1.0),
    ]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["xent_fwd", "xent_bwd", "distill_fwd", "distill_bwd"])
    layout = rng.choice(["nk", "nk", "kn"])
    while True:
        T, V, H = log_uniform(1, 8192), log_uniform(256, 131072), 8 * log_uniform(16, 1024)
        if T * V * H <= 1 << 40:
            break
    if layout == "kn":
        V = V // 8 * 8
    case = {"op": op, "T": T, "V": V, "H": H, "dtype": rng.choice(["bf16", "fp16"]), "layout": layout, "zeta": 0.0,
            "K": 0, "tau": 1.0}
    if op.startswith("xent"):
        case["zeta"] = rng.choice([0.0, 1e-4])
    else:
        case["K"] = min(log_uniform(1, 128), V // 2)
        case["tau"] = rng.choice([1.0, 1.5, 2.0, 4.0])
    return case


def prepare(case, seed):
    T, V, H, K = case["T"], case["V"], case["H"], case["K"]
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    # rows of unit rms and weights that give logits a spread of about 2; a row's
    # target then gets up to 12 more, as a trained model's does
    w = (randn(V, H) * (2.0 / math.sqrt(H))).to(dt)
    x = randn(T, H)
    target = (V * rand(T) ** 2).long().clamp_(max=V - 1)   # low ids are the common words
    x += w[target].float() * (3.0 * rand(T, 1))
    x = x.to(dt)
    s = {"op": case["op"], "x": x, "w": w if case["layout"] == "nk" else w.t().contiguous(), "layout": case["layout"],
         "zeta": case["zeta"], "tau": case["tau"]}
    if case["op"].startswith("xent"):
        if T > 1:
            target = torch.where(rand(T) < 0.05, -100, target)   # prompt and padding rows
        s["target"] = target
    else:
        # distinct entries that start at the target, the teacher's logits falling
        gaps = 1 + (rand(T, K) ** 3 * (V // K - 1)).long()
        gaps[:, 0] = 0
        idx = (target[:, None] + gaps.cumsum(1)) % V
        value = (randn(T, K) * 3.0).sort(dim=1, descending=True).values
        keep = torch.where(rand(T) < 0.1, (rand(T) * (K + 1)).long(), K)   # some rows hold fewer entries, or none
        if T == 2:
            keep = torch.full_like(keep, K)
        idx = torch.where(torch.arange(K, device=DEV) < keep[:, None], idx, -1)
        s["idx"], s["teacher"] = idx, value
    if case["op"].endswith("bwd"):
        # the incoming gradient of each row's loss: a mean in bf16, a scaled sum in fp16
        s["grad"] = (0.5 + rand(T)) / (T if case["dtype"] == "bf16" else 1)
        s["lse"] = _stats(_logits(s), s["tau"])   # saved by the forward pass
    return s


# ---- the plain forms -------------------------------------------------------------
def _logits(s):
    w = s["w"].float()
    return s["x"].float() @ (w.t() if s["layout"] == "nk" else w)


def _stats(z, tau):
    m = z.amax(dim=1, keepdim=True)
    return (((z - m) / tau).exp().sum(dim=1).log() + m[:, 0] / tau)


def _teacher(s):
    """(entries' probabilities with 0 where padded, sum q log q, valid rows)."""
    on = s["idx"] >= 0
    t = torch.where(on, s["teacher"] / s["tau"], -math.inf)
    m = t.amax(dim=1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    e = torch.where(on, (t - m).exp(), 0.0)
    total = e.sum(dim=1, keepdim=True)
    rows = total[:, 0] > 0
    q = e / torch.where(rows[:, None], total, 1.0)
    log_q = torch.where(on, t - m - torch.where(rows[:, None], total, 1.0).log(), 0.0)
    return q, (q * log_q).sum(dim=1), rows


def _products(s, dz):
    """dx and dw from the logits' gradient."""
    dt = s["x"].dtype
    w, x = s["w"].float(), s["x"].float()
    if s["layout"] == "nk":
        return (dz @ w).to(dt), (dz.t() @ x).to(dt)
    return (dz @ w.t()).to(dt), (x.t() @ dz).to(dt)


def _plain(s):
    z, tau = _logits(s), s["tau"]
    if s["op"] == "xent_fwd":
        lse = _stats(z, 1.0)
        rows = s["target"] >= 0
        at = z.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]
        return torch.where(rows, lse - at + s["zeta"] * lse * lse, 0.0), lse
    if s["op"] == "xent_bwd":
        rows = s["target"] >= 0
        lse = s["lse"]
        dz = (z - lse[:, None]).exp() * (1 + 2 * s["zeta"] * lse)[:, None]
        dz.scatter_add_(1, s["target"].clamp(min=0)[:, None], torch.full_like(lse, -1.0)[:, None])
        return _products(s, dz * torch.where(rows, s["grad"], 0.0)[:, None])
    q, entropy, rows = _teacher(s)
    at = s["idx"].clamp(min=0)
    if s["op"] == "distill_fwd":
        lse = _stats(z, tau)
        loss = tau * tau * (entropy - (q * z.gather(1, at)).sum(dim=1) / tau + lse)
        return torch.where(rows, loss, 0.0), lse
    dz = (z / tau - s["lse"][:, None]).exp()
    dz.scatter_add_(1, at, -q)
    return _products(s, dz * (tau * torch.where(rows, s["grad"], 0.0))[:, None])


# ---- the framework's operators ----------------------------------------------------
def _own(s):
    import dense_gemm_work_amd as dg

    if s["op"] == "xent_fwd":
        return dg.linear_cross_entropy(s["x"], s["w"], s["target"], b_layout=s["layout"], z_loss=s["zeta"])
    if s["op"] == "xent_bwd":
        return dg.linear_cross_entropy_backward(s["grad"], s["x"], s["w"], s["target"], s["lse"],
                                                b_layout=s["layout"], z_loss=s["zeta"])
    if s["op"] == "distill_fwd":
        return dg.linear_distill(s["x"], s["w"], s["idx"], s["teacher"], b_layout=s["layout"], temperature=s["tau"])
    return dg.linear_distill_backward(s["grad"], s["x"], s["w"], s["idx"], s["teacher"], s["lse"],
                                      b_layout=s["layout"], temperature=s["tau"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    T, V, H, K = case["T"], case["V"], case["H"], case["K"]
    labels = T * (8 if K == 0 else K * (8 + 4))   # int64 targets, or int64 entries and fp32 teacher logits
    if case["op"].endswith("fwd"):
        # x and w read, loss and lse written; one product
        return {"bytes": 2 * (T + V) * H + labels + 8 * T, "flops": 2 * T * V * H}
    # x, w, lse and the rows' gradients read, dx and dw written; the logits, which
    # were not kept, and the two gradients' products
    return {"bytes": 4 * (T + V) * H + labels + 8 * T, "flops": 6 * T * V * H}


# ---- the definitions in 64 bits ----------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    x, w = s["x"].double(), s["w"].double()
    if s["layout"] == "kn":
        w = w.t()
    tau, V = s["tau"], w.shape[0]
    losses, lses, dxs, dw = [], [], [], None
    step = 2048
    for lo in range(0, x.shape[0], step):
        rows = slice(lo, lo + step)
        xr = x[rows]
        log_p = torch.matmul(xr, w.t()) / tau
        lse = torch.logsumexp(log_p, dim=1)
        log_p -= lse[:, None]
        if s["op"].startswith("xent"):
            y = s["target"][rows]
            q = torch.zeros_like(log_p)
            q[torch.arange(len(y), device=DEV)[y >= 0], y[y >= 0]] = 1.0
            scale = (y >= 0).double()
            extra = s["zeta"]
            plogp = torch.zeros_like(lse)
        else:
            t = s["teacher"][rows].double() / tau
            t = t.masked_fill(s["idx"][rows] < 0, -math.inf)
            qk = torch.nan_to_num(torch.softmax(t, dim=1), nan=0.0)
            q = torch.zeros(len(t), V + 1, dtype=torch.float64, device=DEV)
            i = s["idx"][rows]
            q.scatter_add_(1, torch.where(i < 0, V, i), qk)
            q = q[:, :V]
            scale = (i >= 0).any(dim=1).double()
            extra = 0.0
            plogp = torch.special.xlogy(qk, qk).sum(dim=1)
        if s["op"].endswith("fwd"):
            loss = tau * tau * (plogp - (q * log_p).sum(dim=1)) + extra * lse * lse
            losses.append(loss * scale)
            lses.append(lse)
            continue
        dz = log_p.exp_()
        dz *= (1.0 + 2.0 * extra * lse)[:, None]
        dz -= q
        dz *= (tau * scale * s["grad"][rows].double())[:, None]
        dxs.append(torch.matmul(dz, w))
        part = torch.matmul(dz.t(), xr)
        dw = part if dw is None else dw.add_(part)
    if s["op"].endswith("fwd"):
        return torch.cat(losses), torch.cat(lses)
    return torch.cat(dxs), dw if s["layout"] == "nk" else dw.t().contiguous()
