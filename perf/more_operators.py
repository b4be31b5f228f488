"""Cases of a decode step's MoE layer and of 8-bit integer products: what each reads, computes and returns.

Four kinds of case over three operators:

  layer     a whole mixture-of-experts layer for a few tokens, experts in a
            slot pool: the router's top-k (ties to the lower expert), a softmax
            over the selected logits, and
              out[t] = sum_j w[t, j] W2_e (silu(Wg_e x_t) * (Wu_e x_t)), e = ids[t, j]
            Weights in bf16, in e4m3 with a scale for each 128 x 128, or in
            e2m1 with an e4m3 scale for each 16 and a global scale; activations
            are not quantised.  Routed ids and weights may be given instead of
            logits; an id of -1 is a route that does not count.
  quantize  rows to 8-bit integers with one scale a row:
              s = amax / 127, code = round(127 v / amax), ties to even
  gemm      out[t, n] = xs[t] ws[n] sum_k xq[t, k] wq[n, k]
  linear    quantize (of the rows, or of silu(gate) * up of them) and then gemm

`run` computes them with elementary torch operations in 32 bits (the quotients
next to a rounding border in 64), or, where `own` is set, through the
library's calls.
"""
import math

import torch

own = False

BLK = 128
STD = 0.02             # of the weights
AMAX_MIN = 2.0 ** -100  # a row's amax is taken as at least this


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token through 10 of 512 experts: latency and a stream of weights
        dict(name="layer one token", op="layer", fmt="fp8", T=1, k=10, E=512, H=2048, I=768, logits="f32", skew=0.0,
             drop=0.0),
        # the same with bf16 experts, four times the bytes of 4-bit ones
        dict(name="layer one token bf16", op="layer", fmt="bf16", T=1, k=10, E=512, H=2048, I=768, logits="bf16",
             skew=0.0, drop=0.0),
        # four sequences decoded together, 4-bit experts
        dict(name="layer four tokens nvfp4", op="layer", fmt="nvfp4", T=4, k=10, E=512, H=2048, I=768, logits="f32",
             skew=0.0, drop=0.0),
        # a small layer with hot experts whose routes were chosen elsewhere, some of them masked out: odd sizes
        dict(name="layer given routes", op="layer", fmt="fp8", T=7, k=3, E=61, H=1088, I=704, logits="none", skew=1.1,
             drop=0.2),
        # the largest decode batch of the operator: 135 experts, a stream of 1.3 GB
        dict(name="layer sixteen tokens", op="layer", fmt="bf16", T=16, k=10, E=512, H=2048, I=768, logits="f32",
             skew=0.0, drop=0.0),
        # the shared expert's input for one token: latency alone
        dict(name="quantize one token", op="quantize", T=1, K=2048, dtype="bf16", pad=0),
        # the long prefill's activations: memory traffic alone
        dict(name="quantize long prefill", op="quantize", T=4096, K=2048, dtype="bf16", pad=0),
        # the shared expert's gate and up projection for one token: a stream of weights
        dict(name="gemm one token", op="gemm", T=1, K=2048, N=1536, out="bf16"),
        # the shared expert's down projection for a short prompt that fills no whole tile
        dict(name="gemm short prompt", op="gemm", T=200, K=768, N=2048, out="bf16"),
        # a wide projection over a long prefill: arithmetic alone
        dict(name="gemm long prefill", op="gemm", T=4096, K=4096, N=8192, out="bf16"),
        # the shared expert's second half at decode width: SwiGLU, codes, down projection
        dict(name="linear decode width", op="linear", T=32, K=768, N=2048, act="swiglu", dtype="bf16", out="bf16"),
        # rows and weights that no vector load is aligned to, fp32 in and out
        dict(name="linear odd sizes", op="linear", T=601, K=1999, N=1001, act="none", dtype="f32", out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("layer", "layer", "layer", "quantize", "gemm", "linear"))
    while True:
        if op == "layer":
            E = _log_int(rng, 4, 512)
            c = dict(op=op, fmt=rng.choice(("bf16", "fp8", "nvfp4")), T=_log_int(rng, 1, 16),
                     k=rng.randint(1, min(10, E)), E=E, H=64 * _log_int(rng, 1, 96), I=64 * _log_int(rng, 1, 32),
                     logits=rng.choice(("f32", "f32", "bf16", "none")), skew=rng.choice((0.0, 0.0, 1.1)), drop=0.0)
            if c["logits"] == "none":
                c["drop"] = rng.choice((0.0, 0.1, 0.3))
            if E * c["H"] * c["I"] <= 512 * 2048 * 768 and work(c)["bytes"] <= work(listed()[4])["bytes"]:
                return c
        elif op == "quantize":
            c = dict(op=op, T=_log_int(rng, 1, 4096), K=_log_int(rng, 1, 16384), dtype=rng.choice(("bf16", "f32")),
                     pad=rng.choice((0, 0, 3, 8)))
            if rng.random() < 0.5:
                c["K"] = max(64, c["K"] // 64 * 64)
            if c["T"] * c["K"] <= 4096 * 2048:
                return c
        else:
            c = dict(op=op, T=_log_int(rng, 1, 4096), K=_log_int(rng, 32, 8192), N=_log_int(rng, 32, 8192))
            if op == "linear":
                c["act"], c["dtype"] = rng.choice(("none", "swiglu")), rng.choice(("bf16", "f32"))
            c["out"] = rng.choice(("bf16", "bf16", "f32"))
            if rng.random() < 0.5:
                c["K"], c["N"] = max(64, c["K"] // 64 * 64), max(64, c["N"] // 64 * 64)
            if 1 << 16 <= c["T"] * c["K"] * c["N"] <= 4096 * 4096 * 4096:
                return c


# ----------------------------------------------------------------- prepare
def _rows(T, W, pad, dtype, g, std=1.0):
    """[T, W] rows of a [T, W + pad] buffer; a few columns are much larger than the rest, as activations have."""
    x = torch.randn((T, W + pad), generator=g, device="cuda") * std
    hot = torch.randint(0, W + pad, (max(1, W // 256),), generator=g, device="cuda")
    x[:, hot] *= 8.0
    return x.to(dtype)[:, :W]


def _layout(fmt, H, I):
    """Byte offsets of an expert row's sections: w13 [2I, H] at 0, then w2
    [H, I], and for the 8- and 4-bit formats their scales, in the order and
    with the alignment that the pool's rows have."""
    up = lambda n: cdiv(n, 16) * 16  # noqa: E731
    if fmt == "bf16":
        return dict(w2=4 * I * H, end=6 * I * H)
    if fmt == "fp8":
        hb, ib = cdiv(H, BLK), cdiv(I, BLK)
        w2 = 2 * I * H
        s13 = w2 + H * I
        s2 = s13 + up(8 * ib * hb)
        return dict(w2=w2, s13=s13, s2=s2, end=s2 + up(4 * ib * hb))
    s13 = I * H
    w2 = s13 + I * H // 8
    s2 = w2 + H * I // 2
    gs = s2 + H * I // 16
    return dict(s13=s13, w2=w2, s2=s2, gs=gs, end=gs + 16)


def _fp8_blocks(w):
    """w [..., N, K] fp32 -> e4m3 bytes and fp32 scales [..., ceil(N/128), ceil(K/128)]."""
    N, K = w.shape[-2:]
    nb, kb = cdiv(N, BLK), cdiv(K, BLK)
    p = torch.nn.functional.pad(w, (0, kb * BLK - K, 0, nb * BLK - N)).reshape(*w.shape[:-2], nb, BLK, kb, BLK)
    s = p.abs().amax(dim=(-3, -1)).clamp_min(1e-12) / 448.0
    q = (p / s[..., :, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(*w.shape[:-2], nb * BLK, kb * BLK)[..., :N, :K].contiguous(), s.contiguous()


def _nvfp4(w):
    """w [n, N, K] fp32 -> packed e2m1 [n, N, K/2], e4m3 scales [n, K/64, N, 4] and global scales [n]."""
    n, N, K = w.shape
    gs = w.abs().amax(dim=(1, 2)) / (6.0 * 448.0)
    p = w.reshape(n, N, K // 16, 16)
    s = (p.abs().amax(-1) / (6.0 * gs[:, None, None])).clamp_min(2.0 ** -6).to(torch.float8_e4m3fn)
    r = p / (s.float() * gs[:, None, None])[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(r.abs(), edges).to(torch.uint8) | ((r < 0).to(torch.uint8) << 3)
    code = code.reshape(n, N, K // 2, 2)
    scales = s.view(torch.uint8).reshape(n, N, K // 64, 4).permute(0, 2, 1, 3)
    return code[..., 0] | (code[..., 1] << 4), scales.contiguous(), gs


def _expert_rows(c, n, lay, g):
    """n expert rows as the pool holds them."""
    fmt, H, I = c["fmt"], c["H"], c["I"]
    rows = torch.zeros((n, lay["end"]), dtype=torch.uint8, device="cuda")
    for at, scales, shape, which in ((0, "s13", (n, 2, I, H), 0), (lay["w2"], "s2", (n, H, I), 1)):
        w = torch.randn(shape, generator=g, device="cuda") * STD
        if fmt == "bf16":
            q = w.to(torch.bfloat16).reshape(n, -1).view(torch.uint8)
            s = None
        elif fmt == "fp8":
            q, s = _fp8_blocks(w)
        else:
            q, s, gs = _nvfp4(w.reshape(n, -1, shape[-1]))
            rows[:, lay["gs"] + 4 * which:lay["gs"] + 4 * which + 4] = gs.reshape(n, 1).view(torch.uint8)
        q = q.reshape(n, -1)
        rows[:, at:at + q.shape[1]] = q
        if s is not None:
            s = s.reshape(n, -1).view(torch.uint8)
            rows[:, lay[scales]:lay[scales] + s.shape[1]] = s
    return rows


def _prepare_layer(c, g):
    T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
    lay = _layout(c["fmt"], H, I)
    S = E + 3
    pool = torch.zeros((S, lay["end"]), dtype=torch.uint8, device="cuda")
    e2s = torch.randperm(S, generator=g, device="cuda")[:E].to(torch.int32)
    step = max(1, (1 << 27) // (3 * H * I))
    for e0 in range(0, E, step):
        n = min(E, e0 + step) - e0
        pool[e2s[e0:e0 + n].long()] = _expert_rows(c, n, lay, g)
    logits = torch.randn((T, E), generator=g, device="cuda")
    if c["skew"]:
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        logits -= c["skew"] * torch.log(rank.float())
    st = dict(x=_rows(T, H, 0, torch.bfloat16, g), pool=pool, e2s=e2s)
    if c["logits"] != "none":
        # bf16 logits hold many equal values
        st["logits"] = logits.to(torch.bfloat16) if c["logits"] == "bf16" else logits
    else:
        top = torch.topk(logits, k, dim=1)
        ids = top.indices.to(torch.int32)
        if c["drop"]:
            ids[torch.rand((T, k), generator=g, device="cuda") < c["drop"]] = -1
            ids[T // 2] = -1     # a token without a route
        st["ids"], st["weights"] = ids.contiguous(), torch.softmax(top.values, dim=1)
    return st


def _codes(n, K, g):
    """Rows of 8-bit integers in a buffer whose row stride is a multiple of 16."""
    b = torch.randn((n, cdiv(K, 16) * 16), generator=g, device="cuda") * 42.0
    return b.round().clamp(-127, 127).to(torch.int8)[:, :K]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & ((1 << 62) - 1))
    st = dict(case=dict(c))
    if c["op"] == "layer":
        st.update(_prepare_layer(c, g))
    else:
        T, K = c["T"], c["K"]
        if c["op"] == "gemm":
            st["xq"] = _codes(T, K, g)
            st["xs"] = torch.rand(T, generator=g, device="cuda") * 0.02 + 0.02
        else:
            W = K * (2 if c.get("act") == "swiglu" else 1)
            st["x"] = _rows(T, W, c.get("pad", 0), torch.bfloat16 if c["dtype"] == "bf16" else torch.float32, g)
        if c["op"] != "quantize":
            st["wq"] = _codes(c["N"], K, g)
            st["ws"] = torch.rand(c["N"], generator=g, device="cuda") * 2e-4 + 4e-4
    if own:
        _own_buffers(c, st)
    return st


# --------------------------------------------------------- the library's calls
def _own_buffers(c, st):
    """The outputs, workspaces and views that a user's program keeps."""
    from offloaded_expert_slot_gb300 import oes

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    T = c["T"]
    st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if c["op"] == "layer":
        k, E, H, I = c["k"], c["E"], c["H"], c["I"]
        fmt = dict(bf16=oes.OES_WFMT_BF16, fp8=oes.OES_WFMT_FP8, nvfp4=oes.OES_WFMT_NVFP4)[c["fmt"]]
        pool = st["pool"]
        st["view"] = oes.routed_experts(0, E, st["e2s"], fmt, pool, pool.shape[1], pool.shape[0], H, I)
        if c["logits"] != "none":
            st["ids"], st["weights"] = new((T, k), torch.int32), new((T, k), torch.float32)
        st["bytes"] = oes.moe_layer_few_tokens_workspace_size(st["view"], T, k)
        st["ws_buf"] = new(max(1, st["bytes"]), torch.uint8)
        st["y"] = new((T, H), torch.bfloat16)
        return
    K = c["K"]
    if c["op"] != "gemm":
        st["xq"], st["xs"] = new((T, cdiv(K, 16) * 16), torch.int8)[:, :K], new(T, torch.float32)
    if c["op"] != "quantize":
        st["bytes"] = oes.moe_int8_gemm_workspace_size(T, K, c["N"])
        st["ws_buf"] = new(max(1, st["bytes"]), torch.uint8)
        st["y"] = new((T, c["N"]), torch.bfloat16 if c["out"] == "bf16" else torch.float32)


def _run_own(st):
    from offloaded_expert_slot_gb300 import oes

    c = st["case"]
    T = c["T"]
    if c["op"] == "layer":
        oes.moe_layer_few_tokens(st["view"], st["x"], T, c["k"], st["ids"], st["weights"], st["ws_buf"], st["bytes"],
                                 st["y"], st["status"], logits=st.get("logits"))
        return st["y"] if c["logits"] == "none" else [st["y"], st["ids"], st["weights"]]
    K = c["K"]
    if c["op"] != "gemm":
        act = oes.OES_ACT_SWIGLU if c.get("act") == "swiglu" else oes.OES_ACT_NONE
        oes.moe_int8_quantize(st["x"], st["x"].stride(0), T, K, act, st["xq"], st["xq"].stride(0), st["xs"])
        if c["op"] == "quantize":
            return [st["xq"], st["xs"]]
    oes.moe_int8_gemm(st["xq"], st["xq"].stride(0), st["xs"], T, K, st["wq"], st["wq"].stride(0), st["ws"], c["N"],
                      st["y"], c["N"], st["ws_buf"], st["bytes"], st["status"])
    return st["y"]


# -------------------------------------------------------------- plain forms
def _decode(c, rows, which):
    """Weights of expert rows [n, bytes], 32 bits: which 0 -> [n, 2I, H], 1 -> [n, H, I]."""
    fmt, H, I = c["fmt"], c["H"], c["I"]
    lay = _layout(fmt, H, I)
    n = rows.shape[0]
    N, K = (2 * I, H) if which == 0 else (H, I)
    at, sat = (0, lay.get("s13")) if which == 0 else (lay["w2"], lay.get("s2"))
    if fmt == "bf16":
        return rows[:, at:at + 2 * N * K].contiguous().view(torch.bfloat16).reshape(n, N, K).float()
    if fmt == "fp8":
        halves = 2 if which == 0 else 1
        nb, kb = cdiv(N // halves, BLK), cdiv(K, BLK)
        w = rows[:, at:at + N * K].contiguous().view(torch.float8_e4m3fn).reshape(n, halves, N // halves, K).float()
        s = rows[:, sat:sat + 4 * halves * nb * kb].contiguous().view(torch.float32).reshape(n, halves, nb, kb)
        s = s.repeat_interleave(BLK, -1)[..., :K].repeat_interleave(BLK, -2)[..., :N // halves, :]
        return (w * s).reshape(n, N, K)
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=rows.device)
    b = rows[:, at:at + N * K // 2].reshape(n, N, K // 2)
    w = value[torch.stack((b & 15, b >> 4), dim=-1).long()].reshape(n, N, K // 16, 16)
    s = rows[:, sat:sat + N * K // 16].contiguous().view(torch.float8_e4m3fn).float()
    s = s.reshape(n, K // 64, N, 4).permute(0, 2, 1, 3).reshape(n, N, K // 16)
    g = rows[:, lay["gs"] + 4 * which:lay["gs"] + 4 * which + 4].contiguous().view(torch.float32)
    return (w * s[..., None]).reshape(n, N, K) * g[:, :, None]


def _run_layer(st):
    c = st["case"]
    T, k, H, I = c["T"], c["k"], c["H"], c["I"]
    if c["logits"] != "none":
        v, ids = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)
        v, ids = v[:, :k], ids[:, :k].to(torch.int32)
        p = torch.exp(v - v[:, :1])
        weights = p / p.sum(1, keepdim=True)
    else:
        ids, weights = st["ids"], st["weights"]
    out = torch.zeros((T, H), device="cuda")
    flat = ids.reshape(-1).long()
    present, which = torch.unique(flat, return_inverse=True)
    # every token against every expert that is present, weighted by the route or by nothing
    share = torch.zeros((present.numel(), T), device="cuda")
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    share.index_put_((which, token), weights.reshape(-1) * (flat >= 0), accumulate=True)
    rows = st["pool"][st["e2s"][present.clamp_min(0)].long()]
    w13 = _decode(c, rows, 0)
    h = torch.matmul(w13, st["x"].float().t())                  # [D, 2I, T]
    del w13
    h = h[:, :I] / (1 + torch.exp(-h[:, :I])) * h[:, I:]
    y = torch.matmul(_decode(c, rows, 1), h)                    # [D, H, T]
    out = (y * share[:, None, :]).sum(0).t().to(torch.bfloat16)
    return out if c["logits"] == "none" else [out, ids, weights]


def _quantize_rows(x):
    """x [T, K] fp32 -> codes and scales [T]; the quotients in 64 bits."""
    a = x.abs().amax(-1).clamp_min(AMAX_MIN)
    q = torch.round(x.double() * 127.0 / a.double()[:, None])
    return q.to(torch.int8), a / 127.0


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "layer":
        return _run_layer(state)
    if c["op"] == "gemm":
        q, s = state["xq"], state["xs"]
    else:
        x = state["x"].float()
        if c.get("act") == "swiglu":
            gate, up = x[:, : c["K"]], x[:, c["K"]:]
            x = gate / (1 + torch.exp(-gate)) * up
        q, s = _quantize_rows(x)
        if c["op"] == "quantize":
            return [q, s]
    sums = torch.matmul(q.float(), state["wq"].float().t())
    return (sums * s[:, None] * state["ws"][None, :]).to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)


# --------------------------------------------------------------------- work
def work(case):
    c = case
    T = c["T"]
    if c["op"] == "layer":
        k, E, H, I = c["k"], c["E"], c["H"], c["I"]
        # the experts the chunk is expected to reach: each token takes k of E
        p = [1.0 / E] * E
        if c["skew"]:
            w = [(e + 1) ** -c["skew"] for e in range(E)]
            p = [v / sum(w) for v in w]
        keep = 1.0 - c["drop"]
        reached = sum(1.0 - (1.0 - min(1.0, k * q) * keep) ** T for q in p)
        routing = dict(f32=4 * E, bf16=2 * E, none=0)[c["logits"]] + 8 * k
        return dict(bytes=reached * _layout(c["fmt"], H, I)["end"] + T * (4 * H + routing),
                    flops=6 * T * k * keep * H * I)
    K, v = c["K"], 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "quantize":
        return dict(bytes=T * K * (v + 1) + 4 * T, flops=3 * T * K)
    N = c["N"]
    rows = T * K + 4 * T if c["op"] == "gemm" else T * K * v * (2 if c["act"] == "swiglu" else 1)
    return dict(bytes=rows + N * K + 4 * N + T * N * (2 if c["out"] == "bf16" else 4), flops=2 * T * N * K)


# -------------------------------------------------------------------- exact
def _e2m1_64(nibbles):
    """Sign, two exponent bits (bias 1) and one mantissa bit, as float64."""
    n = nibbles.double()
    m, e = torch.remainder(n, 2), torch.remainder(torch.div(n, 2, rounding_mode="floor"), 4)
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, e - 1))
    return torch.where(nibbles >= 8, -v, v)


def _matrix_64(c, row, which):
    """One expert's matrix from its row of bytes, float64."""
    fmt, H, I = c["fmt"], c["H"], c["I"]
    lay = _layout(fmt, H, I)
    N, K = (2 * I, H) if which == 0 else (H, I)
    at = 0 if which == 0 else lay["w2"]
    if fmt == "bf16":
        return row[at:at + 2 * N * K].view(torch.bfloat16).reshape(N, K).double()
    sat = lay["s13" if which == 0 else "s2"]
    if fmt == "fp8":
        w = row[at:at + N * K].view(torch.float8_e4m3fn).reshape(N, K).double()
        kb = cdiv(K, BLK)
        half = I if which == 0 else H
        s = row[sat:sat + 4 * cdiv(half, BLK) * kb * (N // half)].view(torch.float32).reshape(-1, kb).double()
        for n0 in range(0, N, half):
            for b in range(cdiv(half, BLK)):
                r0, r1 = n0 + b * BLK, n0 + min(half, (b + 1) * BLK)
                w[r0:r1] *= torch.repeat_interleave(s[n0 // half * cdiv(half, BLK) + b], BLK)[:K]
        return w
    b = row[at:at + N * K // 2].reshape(N, K // 2)
    w = torch.empty((N, K), dtype=torch.float64, device=row.device)
    w[:, 0::2], w[:, 1::2] = _e2m1_64(b % 16), _e2m1_64(torch.div(b, 16, rounding_mode="floor"))
    s = row[sat:sat + N * K // 16].view(torch.float8_e4m3fn).double().reshape(K // 64, N, 4)
    for j in range(K // 16):
        w[:, 16 * j:16 * j + 16] *= s[j // 4, :, j % 4, None]
    return w * row[lay["gs"] + 4 * which:lay["gs"] + 4 * which + 4].view(torch.float32).double()


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    T = c["T"]
    if c["op"] == "layer":
        k, H, I = c["k"], c["H"], c["I"]
        if c["logits"] != "none":
            left = st["logits"].double()
            ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
            chosen = torch.empty((T, k), dtype=torch.float64, device="cuda")
            column = torch.arange(c["E"], device="cuda")
            for j in range(k):
                best = left.max(dim=1, keepdim=True).values
                ids[:, j] = torch.where(left == best, column, c["E"]).min(dim=1).values.to(torch.int32)
                chosen[:, j] = best[:, 0]
                left = left.scatter(1, ids[:, j:j + 1].long(), -math.inf)
            weights = torch.softmax(chosen, dim=1)
        else:
            ids, weights = st["ids"], st["weights"].double()
        x = st["x"].double()
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        for e in torch.unique(ids).tolist():
            if e < 0:
                continue
            t, j = torch.nonzero(ids == e, as_tuple=True)
            row = st["pool"][int(st["e2s"][e])]
            a = x[t] @ _matrix_64(c, row, 0).t()
            y = (a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]) @ _matrix_64(c, row, 1).t()
            out.index_add_(0, t, y * weights[t, j][:, None])
        return out if c["logits"] == "none" else [out, ids, weights]
    if c["op"] == "gemm":
        q, s = st["xq"].double(), st["xs"].double()
    else:
        x = st["x"].double()
        if c.get("act") == "swiglu":
            x = x[:, : c["K"]] * torch.sigmoid(x[:, : c["K"]]) * x[:, c["K"]:]
        a = torch.maximum(x.max(dim=1).values, -x.min(dim=1).values).clamp_min(AMAX_MIN)
        q, s = torch.round(x * 127 / a[:, None]), a / 127
        if c["op"] == "quantize":
            return [q.to(torch.int8), s]
    return (q @ st["wq"].double().t()) * s[:, None] * st["ws"].double()
