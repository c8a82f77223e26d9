"""The gated feed-forward block and the projection with low-rank adapters: cases, inputs, plain forms and 64-bit values.

Four operators of a transformer layer's weights, x [T,H] hidden states:

  ffn   forward   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
  ffn   backward  dh = dy Wd, dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu,
                  dWg = dg^T x, dWu = du^T x, dWd = dy^T h
  lora  forward   y_t = x_t W^T + c_a (x_t A_a^T) B_a^T, a the adapter of row t (-1: none)
  lora  backward  ds_t = c_a dy_t B_a, dx_t = dy_t W + ds_t A_a, dA_a = sum ds_t (x) x_t, dB_a = sum dy_t (x) c_a x_t A_a^T

Weights are stored with the input contiguous ("nk", as written above) or with
the output contiguous ("kn", each matrix transposed).

Where `own` is false `run` computes them with elementary torch operations in
fp32; where it is true it calls dense_gemm_work_amd.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    def ffn(name, op, T, H, F, dtype="bf16", layout="nk", act="silu", save=False):
        return {"name": name, "op": op, "T": T, "H": H, "F": F, "dtype": dtype, "layout": layout, "act": act, "save": save}

    def lora(name, op, T, H, N, L, R, requests, dtype="bf16", layout="nk"):
        return {"name": name, "op": op, "T": T, "H": H, "N": N, "L": L, "R": R, "requests": requests, "dtype": dtype,
                "layout": layout}

    return [
        # one token's decoding step in a small model: latency
        ffn("ffn fwd 1 token", "ffn_fwd", 1, 1536, 4096),
        # a decoding step of a batch of requests: the weights' stream
        ffn("ffn fwd 48 tokens", "ffn_fwd", 48, 4096, 12288, "fp16"),
        # the forward pass of a ragged micro-batch, weights stored with the output contiguous, gate and up kept
        ffn("ffn fwd 777 tokens", "ffn_fwd", 777, 2048, 5632, layout="kn", act="gelu", save=True),
        # a long prompt
        ffn("ffn fwd 8192 tokens", "ffn_fwd", 8192, 4096, 12288),
        # fine-tuning on one short answer, a hidden size that no tile divides
        ffn("ffn bwd 331 tokens", "ffn_bwd", 331, 1536, 4104, "fp16", act="gelu"),
        # an ordinary training micro-batch
        ffn("ffn bwd 2048 tokens", "ffn_bwd", 2048, 2048, 8192),
        # the largest: a long micro-batch
        ffn("ffn bwd 8192 tokens", "ffn_bwd", 8192, 4096, 12288),
        # one token's decoding step with an adapter: latency
        lora("lora fwd 1 token", "lora_fwd", 1, 2048, 2048, 8, 16, 1),
        # a decoding step of many requests, each with an adapter of its own choice
        lora("lora fwd 96 tokens", "lora_fwd", 96, 4096, 4096, 64, 16, 96),
        # prompts of many requests, packed
        lora("lora fwd 5000 tokens", "lora_fwd", 5000, 4096, 8192, 24, 64, 29, "fp16"),
        # adapters of one user's data trained on short answers
        lora("lora bwd 512 tokens", "lora_bwd", 512, 2048, 4096, 1, 8, 4, layout="kn"),
        # several users' adapters trained at once
        lora("lora bwd 8192 tokens", "lora_bwd", 8192, 4096, 4096, 8, 64, 32),
    ]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ffn_fwd", "ffn_bwd", "lora_fwd", "lora_bwd"])
    common = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "layout": rng.choice(["nk", "nk", "kn"])}
    T = log_uniform(1 if op.endswith("fwd") else 16, 8192)
    if op.startswith("ffn"):
        return dict(common, T=T, H=8 * log_uniform(16, 512), F=8 * log_uniform(32, 1536), act=rng.choice(["silu", "silu", "gelu"]),
                    save=op == "ffn_fwd" and rng.choice([False, True]))
    L, R = log_uniform(1, 64), 8 * log_uniform(1, 16)
    L = min(L, max(1, 4096 // R))
    requests = min(T, log_uniform(1, 64)) if T > 256 else T
    return dict(common, T=T, H=8 * log_uniform(32, 512), N=8 * log_uniform(32, 1024), L=L, R=R, requests=requests)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt, nk = DTYPES[case["dtype"]], case["layout"] == "nk"

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def weight(*shape, gain=1.0):
        """[..., out, in] with outputs of the inputs' size, as the layout stores it."""
        w = (randn(*shape) * (gain / math.sqrt(shape[-1]))).to(dt)
        return w if nk else w.transpose(-1, -2).contiguous()

    T, H = case["T"], case["H"]
    # hidden states after a norm: rows of unit size, a few features larger than the rest
    x = randn(T, H)
    x[:, :: max(1, H // 8)] *= 4.0
    s = {"op": case["op"], "layout": case["layout"], "x": x.to(dt)}
    if case["op"].startswith("ffn"):
        F = case["F"]
        s.update(act=case["act"], save=case["save"], w_gate=weight(F, H, gain=1.5), w_up=weight(F, H), w_down=weight(H, F))
        if case["op"] == "ffn_bwd":
            s["dy"] = (randn(T, H) * (0.01 if case["dtype"] == "bf16" else 1.0)).to(dt)   # fp16: a scaled loss
            # what the forward pass kept
            s["gate"], s["up"] = (s["x"] @ (w.t() if nk else w) for w in (s["w_gate"], s["w_up"]))
        return s
    N, L, R, requests = case["N"], case["L"], case["R"], case["requests"]
    s.update(w=weight(N, H), a=weight(L, R, H), b=weight(L, N, R, gain=0.5))
    s["scale"] = 0.5 + torch.rand(L, generator=g, device=DEV)
    # requests of uneven lengths one after the other, one in ten without an adapter
    owner = torch.randint(0, L, (requests,), generator=g, device=DEV)
    owner[torch.rand(requests, generator=g, device=DEV) < 0.1] = -1
    if requests <= 4:
        owner[0] = 0
    cuts = torch.randperm(T - 1, generator=g, device=DEV)[: requests - 1] + 1
    of = torch.zeros(T, dtype=torch.int64, device=DEV)
    of[cuts] = 1
    s["adapter"] = owner[of.cumsum(0)]
    if case["op"] == "lora_bwd":
        s["dy"] = (randn(T, N) * (0.01 if case["dtype"] == "bf16" else 1.0)).to(dt)
    return s


# ---- the plain forms -------------------------------------------------------------
def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        p = 1.0 / (1.0 + (-g).exp())
        return g * p, p * (1.0 + g * (1.0 - p))
    phi = 0.5 * (1.0 + torch.erf(g / math.sqrt(2.0)))
    return g * phi, phi + g * (g * g * -0.5).exp() / math.sqrt(2.0 * math.pi)


def _plain_ffn(s):
    dt, nk = s["x"].dtype, s["layout"] == "nk"
    x = s["x"].float()
    wg, wu, wd = (s[n].float() if nk else s[n].float().t() for n in ("w_gate", "w_up", "w_down"))
    if s["op"] == "ffn_fwd":
        g, u = x @ wg.t(), x @ wu.t()
        y = ((_act(g, s["act"])[0] * u) @ wd.t()).to(dt)
        return (y, g.to(dt), u.to(dt)) if s["save"] else y
    g, u, dy = s["gate"].float(), s["up"].float(), s["dy"].float()
    a, slope = _act(g, s["act"])
    dh = dy @ wd
    dg, du = dh * u * slope, dh * a
    dx = dg @ wg + du @ wu
    if nk:
        dws = dg.t() @ x, du.t() @ x, dy.t() @ (a * u)
    else:
        dws = x.t() @ dg, x.t() @ du, (a * u).t() @ dy
    return (dx.to(dt), *(d.to(dt) for d in dws))


def _plain_lora(s):
    dt, nk = s["x"].dtype, s["layout"] == "nk"
    x = s["x"].float()
    w, a, b = (s[n].float() if nk else s[n].float().transpose(-1, -2) for n in ("w", "a", "b"))
    L, R, H = a.shape
    a = a.reshape(L * R, H)                               # all adapters side by side
    b = b.transpose(0, 1).reshape(-1, L * R)
    own_columns = s["adapter"][:, None] == torch.arange(L, device=x.device)
    mask = (own_columns * s["scale"]).repeat_interleave(R, dim=1)
    if s["op"] == "lora_fwd":
        return (x @ w.t() + (x @ a.t() * mask) @ b.t()).to(dt)
    dy = s["dy"].float()
    ds = dy @ b * mask
    dx = dy @ w + ds @ a
    if nk:
        da = (ds.t() @ x).reshape(L, R, H)
        db = (dy.t() @ (x @ a.t() * mask)).reshape(-1, L, R).transpose(0, 1)
    else:
        da = (x.t() @ ds).reshape(H, L, R).transpose(0, 1)
        db = ((x @ a.t() * mask).t() @ dy).reshape(L, R, -1)
    return dx.to(dt), da.to(dt).contiguous(), db.to(dt).contiguous()


# ---- the framework's operators ----------------------------------------------------
def _own(s):
    import dense_gemm_work_amd as dg

    if s["op"] == "ffn_fwd":
        return dg.gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], activation=s["act"], b_layout=s["layout"],
                            save=s["save"])
    if s["op"] == "ffn_bwd":
        return dg.gated_ffn_backward(s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"], s["up"],
                                     activation=s["act"], b_layout=s["layout"])
    if s["op"] == "lora_fwd":
        return dg.linear_lora(s["x"], s["w"], s["a"], s["b"], s["adapter"], scale=s["scale"], b_layout=s["layout"])
    return dg.linear_lora_backward(s["dy"], s["x"], s["w"], s["a"], s["b"], s["adapter"], scale=s["scale"],
                                   b_layout=s["layout"])


def run(state):
    if own:
        return _own(state)
    return _plain_ffn(state) if state["op"].startswith("ffn") else _plain_lora(state)


def work(case):
    T, H = case["T"], case["H"]
    if case["op"].startswith("ffn"):
        F = case["F"]
        if case["op"] == "ffn_fwd":
            # x and the three weights read, y (and gate and up) written; three products
            return {"bytes": 2 * (2 * T * H + 3 * H * F + (2 * T * F if case["save"] else 0)), "flops": 6 * T * H * F}
        # x, dy, gate, up and the weights read, dx and the weights' gradients written; six products
        return {"bytes": 2 * (3 * T * H + 2 * T * F + 6 * H * F), "flops": 12 * T * H * F}
    N, L, R = case["N"], case["L"], case["R"]
    used = min(L, case["requests"])   # adapters that a call can meet
    if case["op"] == "lora_fwd":
        return {"bytes": 2 * (T * H + T * N + H * N + used * R * (H + N)) + 8 * T + 4 * L,
                "flops": 2 * T * H * N + 2 * T * R * (H + N)}
    # x, dy, w and the used adapters read; dx and every adapter's gradients written
    return {"bytes": 2 * (2 * T * H + T * N + H * N + (used + L) * R * (H + N)) + 8 * T + 4 * L,
            "flops": 2 * T * H * N + 6 * T * R * (H + N) - 2 * T * R * N}


# ---- the definitions in 64 bits ----------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and k != "adapter"}
    if case["layout"] == "kn":
        for k in ("w_gate", "w_up", "w_down", "w", "a", "b"):
            if k in f:
                f[k] = f[k].transpose(-1, -2)

    def stored(w):
        return w if case["layout"] == "nk" else w.transpose(-1, -2).contiguous()

    x = f["x"]
    if case["op"].startswith("ffn"):
        fn = torch.nn.functional.silu if case["act"] == "silu" else torch.nn.functional.gelu
        if case["op"] == "ffn_fwd":
            g, u = torch.matmul(x, f["w_gate"].t()), torch.matmul(x, f["w_up"].t())
            y = torch.matmul(fn(g) * u, f["w_down"].t())
            return (y, g, u) if case["save"] else y
        with torch.enable_grad():
            g, u = f["gate"].requires_grad_(), f["up"].requires_grad_()
            h = fn(g) * u
        dg, du = torch.autograd.grad(h, (g, u), torch.matmul(f["dy"], f["w_down"]))
        dx = torch.matmul(dg, f["w_gate"]) + torch.matmul(du, f["w_up"])
        return (dx, stored(torch.matmul(dg.t(), x)), stored(torch.matmul(du.t(), x)),
                stored(torch.matmul(f["dy"].t(), h.detach())))
    w, a, b = f["w"], f["a"], f["b"]
    if case["op"] == "lora_fwd":
        y = torch.matmul(x, w.t())
    else:
        dy = f["dy"]
        dx, da, db = torch.matmul(dy, w), torch.zeros_like(a), torch.zeros_like(b)
    for i in range(a.shape[0]):
        rows = torch.nonzero(s["adapter"] == i)[:, 0]
        low = torch.matmul(x[rows], a[i].t()) * f["scale"][i]
        if case["op"] == "lora_fwd":
            y[rows] += torch.matmul(low, b[i].t())
            continue
        dlow = torch.matmul(dy[rows], b[i]) * f["scale"][i]
        dx[rows] += torch.matmul(dlow, a[i])
        da[i] = torch.matmul(dlow.t(), x[rows])
        db[i] = torch.matmul(dy[rows].t(), low)
    return y if case["op"] == "lora_fwd" else (dx, stored(da), stored(db))
