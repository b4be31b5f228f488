"""Cases of the operators around 8-bit expert layers: what each reads, computes and returns.

Four operators, one set: an MoE block whose experts and shared expert hold
8-bit (e4m3) weights with one fp32 scale for each block of 128 x 128.

  norm      the residual update after a block and the norm before the next:
              v  = y * rsqrt(mean(y^2) + eps) * (w_offset + w_post)
              r' = residual + residual_scale * gate * v
              u  = r' * rsqrt(mean(r'^2) + eps) * (w_offset + w_pre)
            and u in 8 bits, one scale for each 128 values of a row
  quantize  rows to 8 bits: over each 128 values s = amax / 448 and codes
            e4m3(448 x / amax); optionally of silu(gate) * up
  gemm      out = x @ w^T of 8-bit rows, x with a scale for each 1 x 128, w
            for each 128 x 128
  experts   the expert layer over a slot pool, routed tokens grouped by
            expert: out[t] = sum_j weights[t, j] * mlp_{ids[t, j]}(x[t]),
            mlp(x) = q(silu(q(x) gate^T) * (q(x) up^T)) w2^T with q the
            quantiser above

`run` computes them with elementary torch operations in 32 bits, or, where
`own` is set, through the library's calls.
"""
import math

import torch

own = False

CODE_MAX = 448.0        # largest e4m3 value
AMAX_MIN = 2.0 ** -100  # a group's amax is taken as at least this
BLK = 128
EPS = 1e-6
W_OFFSET = 0.0
RESIDUAL_SCALE = 0.5
STD = 0.02              # of the weights


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the step between two blocks for one decoded token: latency alone
        dict(name="norm decode", op="norm", T=1, H=2048, res="bf16", gate="token", quant=True, pad=0),
        # a ragged chunk over an odd width, an fp32 residual stream, a learned
        # scale per channel: rows that no vector load is aligned to
        dict(name="norm odd width", op="norm", T=601, H=1999, res="f32", gate="channel", quant=False, pad=0),
        # the long prefill's chunk: memory traffic alone
        dict(name="norm long prefill", op="norm", T=4096, H=2048, res="bf16", gate="token", quant=True, pad=0),
        # the shared expert's hidden rows at decode width, SwiGLU fused
        dict(name="quantize swiglu decode", op="quantize", T=32, K=768, act="swiglu", dtype="bf16", pad=0),
        # the long prefill's activations
        dict(name="quantize long prefill", op="quantize", T=4096, K=2048, act="none", dtype="bf16", pad=0),
        # the shared expert's gate and up projection for one token: a stream of weights
        dict(name="gemm one token", op="gemm", T=1, K=2048, N=1536, out="bf16"),
        # the shared expert's down projection for a short prompt that fills no whole tile
        dict(name="gemm short prompt", op="gemm", T=200, K=768, N=2048, out="bf16"),
        # a wide projection over a long prefill: arithmetic alone
        dict(name="gemm long prefill", op="gemm", T=4096, K=4096, N=8192, out="bf16"),
        # one decoded token through 10 of 512 experts
        dict(name="experts one token", op="experts", T=1, k=10, E=512, H=2048, I=768, skew=0.0, drop=0.0),
        # decode width: about one route an expert, a stream of half the layer
        dict(name="experts decode width", op="experts", T=32, k=10, E=512, H=2048, I=768, skew=0.0, drop=0.0),
        # a prefill chunk whose router has hot experts: ragged groups, and some routes masked out
        dict(name="experts skewed prefill", op="experts", T=600, k=10, E=512, H=2048, I=768, skew=1.1, drop=0.05),
        # the long prefill's chunk: every expert, 80 routes each
        dict(name="experts long prefill", op="experts", T=4096, k=10, E=512, H=2048, I=768, skew=0.0, drop=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "quantize", "gemm", "gemm", "experts", "experts"))
    while True:
        if op == "norm":
            c = dict(op=op, T=_log_int(rng, 1, 4096), H=_log_int(rng, 64, 8192), res=rng.choice(("bf16", "f32")),
                     gate=rng.choice(("none", "token", "channel", "element")), quant=rng.random() < 0.5,
                     pad=rng.choice((0, 0, 3, 8)))
            if rng.random() < 0.5:
                c["H"] = max(64, c["H"] // 64 * 64)
            if c["T"] * c["H"] <= 4096 * 2048:
                return c
        elif op == "quantize":
            c = dict(op=op, T=_log_int(rng, 1, 4096), K=_log_int(rng, 64, 8192), act=rng.choice(("none", "swiglu")),
                     dtype=rng.choice(("bf16", "f32")), pad=rng.choice((0, 0, 3, 8)))
            if rng.random() < 0.5:
                c["K"] = max(64, c["K"] // 64 * 64)
            if c["T"] * c["K"] <= 4096 * 2048:
                return c
        elif op == "gemm":
            c = dict(op=op, T=_log_int(rng, 1, 4096), K=_log_int(rng, 100, 8192), N=_log_int(rng, 100, 8192),
                     out=rng.choice(("bf16", "bf16", "f32")))
            if rng.random() < 0.5:
                c["K"], c["N"] = max(128, c["K"] // 64 * 64), max(64, c["N"] // 64 * 64)
            if 1 << 16 <= c["T"] * c["K"] * c["N"] <= 4096 * 4096 * 8192:
                return c
        else:
            E = _log_int(rng, 8, 512)
            c = dict(op=op, T=_log_int(rng, 1, 4096), k=rng.randint(1, min(10, E)), E=E,
                     H=64 * _log_int(rng, 2, 64), I=64 * _log_int(rng, 1, 24), skew=rng.choice((0.0, 0.0, 1.1)),
                     drop=rng.choice((0.0, 0.0, 0.05)))
            if c["T"] * c["k"] * c["H"] * c["I"] <= 40960 * 2048 * 768 and E * c["H"] * c["I"] <= 512 * 2048 * 768:
                return c


# ----------------------------------------------------------------- prepare
def _rows(T, W, pad, dtype, g, std=1.0):
    """[T, W] rows of a [T, W + pad] buffer; a few columns are much larger than the rest, as activations have."""
    x = torch.randn((T, W + pad), generator=g, device="cuda") * std
    hot = torch.randint(0, W + pad, (max(1, W // 256),), generator=g, device="cuda")
    x[:, hot] *= 8.0
    return x.to(dtype)[:, :W]


def _quantize_blocks(w):
    """w [..., N, K] fp32 -> e4m3 codes and fp32 scales [..., ceil(N/128), ceil(K/128)] for each 128 x 128."""
    N, K = w.shape[-2:]
    nb, kb = cdiv(N, BLK), cdiv(K, BLK)
    p = torch.nn.functional.pad(w, (0, kb * BLK - K, 0, nb * BLK - N))
    p = p.reshape(*w.shape[:-2], nb, BLK, kb, BLK)
    s = p.abs().amax(dim=(-3, -1)).clamp_min(1e-12) / CODE_MAX
    q = (p / s[..., :, None, :, None]).clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(*w.shape[:-2], nb * BLK, kb * BLK)[..., :N, :K].contiguous()
    return q, s.contiguous()


def _pad16(q):
    """Rows of bytes in a buffer whose row stride is a multiple of 16."""
    ld = cdiv(q.shape[1], 16) * 16
    b = torch.zeros((q.shape[0], ld), dtype=torch.uint8, device=q.device)
    b[:, : q.shape[1]] = q
    return b[:, : q.shape[1]]


def _row_layout(H, I):
    """Byte offsets of an expert row: w13 [2I, H], w2 [H, I] e4m3; w13 scales
    [2 ceil(I/128), ceil(H/128)] (gate, then up), w2 scales [ceil(H/128), ceil(I/128)] fp32."""
    hb, ib = cdiv(H, BLK), cdiv(I, BLK)
    w2 = 2 * I * H
    s13 = w2 + H * I
    s2 = s13 + cdiv(2 * ib * hb * 4, 16) * 16
    return dict(w2=w2, s13=s13, s2=s2, end=s2 + cdiv(hb * ib * 4, 16) * 16, hb=hb, ib=ib)


def _prepare_experts(c, g):
    T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
    lay = _row_layout(H, I)
    hb, ib = lay["hb"], lay["ib"]
    S = E + 3
    pool = torch.zeros((S, lay["end"]), dtype=torch.uint8, device="cuda")
    e2s = torch.randperm(S, generator=g, device="cuda")[:E].to(torch.int32)
    step = max(1, (1 << 26) // (3 * H * I))
    for e0 in range(0, E, step):
        n = min(E, e0 + step) - e0
        slots = e2s[e0:e0 + n].long()
        rows = torch.zeros((n, lay["end"]), dtype=torch.uint8, device="cuda")
        q, s = _quantize_blocks(torch.randn((n, 2, I, H), generator=g, device="cuda") * STD)
        rows[:, : lay["w2"]] = q.reshape(n, -1)
        rows[:, lay["s13"]:lay["s13"] + 8 * ib * hb] = s.reshape(n, -1).view(torch.uint8)
        q, s = _quantize_blocks(torch.randn((n, H, I), generator=g, device="cuda") * STD)
        rows[:, lay["w2"]:lay["s13"]] = q.reshape(n, -1)
        rows[:, lay["s2"]:lay["s2"] + 4 * ib * hb] = s.reshape(n, -1).view(torch.uint8)
        pool[slots] = rows
    logits = torch.randn((T, E), generator=g, device="cuda")
    if c["skew"]:
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        logits -= c["skew"] * torch.log(rank.float())
    top = torch.topk(logits, k, dim=1)
    ids = top.indices.to(torch.int32)
    if c["drop"]:
        ids[torch.rand((T, k), generator=g, device="cuda") < c["drop"]] = -1
    st = dict(x=_rows(T, H, 0, torch.bfloat16, g), ids=ids.contiguous(), weights=torch.softmax(top.values, dim=1),
              pool=pool, e2s=e2s)
    # the most routes one expert has: the plain form's rows for each expert
    st["most"] = max(1, int(torch.bincount(ids[ids >= 0].long(), minlength=E).max()))
    if own:
        _own_experts(c, st)
    return st


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & ((1 << 62) - 1))
    st = dict(case=dict(c))
    if c["op"] == "norm":
        T, H, pad = c["T"], c["H"], c["pad"]
        st["residual"] = _rows(T, H, pad, torch.bfloat16 if c["res"] == "bf16" else torch.float32, g, 4.0)
        st["y"] = _rows(T, H, pad, torch.bfloat16, g)
        st["post"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        st["pre"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        gate = c["gate"]
        if gate == "token":      # logits of one sigmoid gate a token
            st["gate"] = torch.randn(T, generator=g, device="cuda")
        elif gate == "channel":  # a learned scale, used as it stands
            st["gate"] = torch.rand(H, generator=g, device="cuda").to(torch.bfloat16)
        elif gate == "element":  # logits of a gate for each value
            st["gate"] = _rows(T, H, pad, torch.bfloat16, g)
    elif c["op"] == "quantize":
        st["x"] = _rows(c["T"], c["K"] * (2 if c["act"] == "swiglu" else 1), c["pad"],
                        torch.bfloat16 if c["dtype"] == "bf16" else torch.float32, g)
    elif c["op"] == "gemm":
        T, K, N = c["T"], c["K"], c["N"]
        x = _rows(T, K, 0, torch.float32, g)
        s = torch.nn.functional.pad(x, (0, cdiv(K, BLK) * BLK - K)).reshape(T, -1, BLK).abs().amax(-1) / CODE_MAX
        st["xs"] = s.contiguous()
        q = (x / s.repeat_interleave(BLK, 1)[:, :K]).clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn)
        st["xq"] = _pad16(q.view(torch.uint8))
        q, st["ws"] = _quantize_blocks(torch.randn((N, K), generator=g, device="cuda") * STD)
        st["wq"] = _pad16(q)
    else:
        st.update(_prepare_experts(c, g))
    if own and c["op"] != "experts":
        _own_buffers(c, st)
    return st


# --------------------------------------------------------- the library's calls
def _own_buffers(c, st):
    """The output buffers a user's program keeps, and the argument block of the norm."""
    from offloaded_expert_slot_gb300 import oes

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    T = c["T"]
    if c["op"] == "norm":
        H = c["H"]
        st["r_out"] = new((T, H), st["residual"].dtype)
        st["u"] = new((T, H), torch.bfloat16)
        if c["quant"]:
            st["q"], st["s"] = new((T, H), torch.uint8), new((T, cdiv(H, BLK)), torch.float32)
        kind = dict(none=oes.OES_GATE_NONE, token=oes.OES_GATE_TOKEN, channel=oes.OES_GATE_CHANNEL,
                    element=oes.OES_GATE_ELEMENT)[c["gate"]]
        st["args"] = oes.block_norm(
            T, H, st["residual"], residual_ld=st["residual"].stride(0), y=st["y"], y_ld=st["y"].stride(0),
            post_weight=st["post"], pre_weight=st["pre"], gate=st.get("gate"), gate_kind=kind,
            gate_ld=st["gate"].stride(0) if c["gate"] in ("token", "element") else 0,
            gate_sigmoid=c["gate"] in ("token", "element"), residual_scale=RESIDUAL_SCALE, weight_offset=W_OFFSET,
            eps=EPS, out_residual=st["r_out"], out=st["u"], out_q=st.get("q"), out_scale=st.get("s"))
    elif c["op"] == "quantize":
        st["q"], st["s"] = new((T, c["K"]), torch.uint8), new((T, cdiv(c["K"], BLK)), torch.float32)
    else:
        st["out"] = new((T, c["N"]), torch.bfloat16 if c["out"] == "bf16" else torch.float32)
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def _own_experts(c, st):
    """The view of the pool, the workspaces and the align's outputs a user's program keeps."""
    from offloaded_expert_slot_gb300 import oes

    T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
    R, pool = T * k, st["pool"]

    def new(n, dtype):
        return torch.empty(max(1, n), dtype=dtype, device="cuda")

    B = st["B"] = oes.oes_tile_plan(R, E)
    cap = oes.align_capacity(R, E, B)
    st["view"] = oes.routed_experts(0, E, st["e2s"], oes.OES_WFMT_FP8, pool, pool.shape[1], pool.shape[0], H, I)
    st["sorted"], st["blocks"], st["npad"] = new(cap, torch.int32), new(cap // B, torch.int32), new(1, torch.int32)
    st["align_bytes"] = oes.moe_align_workspace_size(R, E, B)
    st["align_ws"] = new(st["align_bytes"], torch.uint8)
    st["gemm_bytes"] = oes.moe_grouped_gemm_workspace_size(st["view"], T, k)
    st["gemm_ws"] = new(st["gemm_bytes"], torch.uint8)
    st["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def _run_own(st):
    from offloaded_expert_slot_gb300 import oes

    c = st["case"]
    T = c["T"]
    if c["op"] == "norm":
        oes.moe_block_norm(st["args"])
        out = [st["r_out"], st["u"]]
        if c["quant"]:
            out += [st["q"].view(torch.float8_e4m3fn), st["s"]]
        return out
    if c["op"] == "quantize":
        act = oes.OES_ACT_SWIGLU if c["act"] == "swiglu" else oes.OES_ACT_NONE
        oes.moe_fp8_quantize(st["x"], st["x"].stride(0), T, c["K"], act, st["q"], c["K"], st["s"])
        return [st["q"].view(torch.float8_e4m3fn), st["s"]]
    if c["op"] == "gemm":
        oes.moe_fp8_gemm(st["xq"], st["xq"].stride(0), st["xs"], T, c["K"], st["wq"], st["wq"].stride(0), st["ws"],
                         c["N"], st["out"], c["N"], st["status"])
        return st["out"]
    R = T * c["k"]
    oes.moe_align_block_size(st["ids"], R, c["E"], st["B"], 1, st["sorted"], st["blocks"], st["npad"], st["status"],
                             st["align_ws"], st["align_bytes"])
    oes.moe_grouped_gemm_slots(st["view"], st["x"], T, c["k"], st["ids"], st["weights"], st["sorted"], st["blocks"],
                               st["npad"], st["B"], st["gemm_ws"], st["gemm_bytes"], st["out"], st["status"])
    return st["out"]


# -------------------------------------------------------------- plain forms
def _f8(b):
    return b.view(torch.float8_e4m3fn).float()


def _quantize_rows(x):
    """x [..., K] fp32 -> codes as e4m3 and scales [..., ceil(K/128)]."""
    K = x.shape[-1]
    p = torch.nn.functional.pad(x, (0, cdiv(K, BLK) * BLK - K)).reshape(*x.shape[:-1], -1, BLK)
    a = torch.where(torch.isnan(p), 0.0, p.abs()).amax(-1).clamp_min(AMAX_MIN)
    q = (p * CODE_MAX / a[..., None]).clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn)
    return q.reshape(*x.shape[:-1], -1)[..., :K].contiguous(), a / CODE_MAX


def _dequantize_rows(q, s):
    return q.float() * s.repeat_interleave(BLK, -1)[..., : q.shape[-1]]


def _dequantize_blocks(b, s):
    """codes [..., N, K] bytes and scales for each 128 x 128 -> fp32."""
    N, K = b.shape[-2:]
    full = s.repeat_interleave(BLK, -1)[..., :K].repeat_interleave(BLK, -2)[..., :N, :]
    return _f8(b.contiguous()) * full


def _run_norm(st):
    c = st["case"]

    def norm(v, w):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * (W_OFFSET + w.float())

    v = norm(st["y"].float(), st["post"])
    if c["gate"] == "token":
        v = v * torch.sigmoid(st["gate"].float())[:, None]
    elif c["gate"] == "channel":
        v = v * st["gate"].float()
    elif c["gate"] == "element":
        v = v * torch.sigmoid(st["gate"].float())
    r = st["residual"].float() + RESIDUAL_SCALE * v
    u = norm(r, st["pre"])
    out = [r.to(st["residual"].dtype), u.to(torch.bfloat16)]
    return out + list(_quantize_rows(u)) if c["quant"] else out


def _run_experts(st):
    c = st["case"]
    T, k, H, I = c["T"], c["k"], c["H"], c["I"]
    lay = _row_layout(H, I)
    hb, ib = lay["hb"], lay["ib"]
    flat = st["ids"].reshape(-1).long()
    route = torch.nonzero(flat >= 0).reshape(-1)                  # the routes that count
    present, which = torch.unique(flat[route], return_inverse=True)
    order = torch.argsort(which, stable=True)
    first = torch.cumsum(torch.bincount(which), 0) - torch.bincount(which)
    which, route = which[order], route[order]
    place = torch.arange(route.numel(), device=flat.device) - first[which]
    rows = st["pool"][st["e2s"][present].long()]
    D = present.numel()
    x = _dequantize_rows(*_quantize_rows(st["x"].float()))
    xs = torch.zeros((D, st["most"], H), device="cuda")
    xs[which, place] = x[route // k]
    s13 = rows[:, lay["s13"]:lay["s13"] + 8 * ib * hb].contiguous().view(torch.float32).reshape(D, 2, ib, hb)
    w13 = _dequantize_blocks(rows[:, : lay["w2"]].reshape(D, 2, I, H), s13)
    gate = torch.bmm(xs, w13[:, 0].transpose(1, 2))
    up = torch.bmm(xs, w13[:, 1].transpose(1, 2))
    h = _dequantize_rows(*_quantize_rows(gate / (1 + torch.exp(-gate)) * up))
    s2 = rows[:, lay["s2"]:lay["s2"] + 4 * ib * hb].contiguous().view(torch.float32).reshape(D, hb, ib)
    w2 = _dequantize_blocks(rows[:, lay["w2"]:lay["s13"]].reshape(D, H, I), s2)
    y = torch.zeros((T * k, H), device="cuda")
    y[route] = torch.bmm(h, w2.transpose(1, 2))[which, place]
    return (y.reshape(T, k, H) * st["weights"][:, :, None]).sum(1).to(torch.bfloat16)


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "norm":
        return _run_norm(state)
    if c["op"] == "quantize":
        x = state["x"].float()
        if c["act"] == "swiglu":
            gate, up = x[:, : c["K"]], x[:, c["K"]:]
            x = gate / (1 + torch.exp(-gate)) * up
        return list(_quantize_rows(x))
    if c["op"] == "gemm":
        x = _dequantize_rows(state["xq"].contiguous().view(torch.float8_e4m3fn), state["xs"])
        w = _dequantize_blocks(state["wq"], state["ws"])
        return torch.matmul(x, w.t()).to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    return _run_experts(state)


# --------------------------------------------------------------------- work
def work(case):
    c = case
    T = c["T"]
    if c["op"] == "norm":
        H, r = c["H"], 2 if c["res"] == "bf16" else 4
        gate = dict(none=0, token=4 * T, channel=2 * H, element=2 * T * H)[c["gate"]]
        b = T * H * (2 * r + 2 + 2) + 4 * H + gate + (T * (H + 4 * cdiv(H, BLK)) if c["quant"] else 0)
        return dict(bytes=b, flops=12 * T * H)
    if c["op"] == "quantize":
        n = T * c["K"]
        return dict(bytes=n * (2 if c["act"] == "swiglu" else 1) * (2 if c["dtype"] == "bf16" else 4) + n
                    + 4 * T * cdiv(c["K"], BLK), flops=4 * n)
    if c["op"] == "gemm":
        K, N = c["K"], c["N"]
        kb = cdiv(K, BLK)
        return dict(bytes=T * K + N * K + 4 * kb * (T + cdiv(N, BLK)) + T * N * (2 if c["out"] == "bf16" else 4),
                    flops=2 * T * N * K)
    k, E, H, I = c["k"], c["E"], c["H"], c["I"]
    # the experts the chunk is expected to reach: each token takes k of E
    p = [1.0 / E] * E
    if c["skew"]:
        w = [(e + 1) ** -c["skew"] for e in range(E)]
        p = [v / sum(w) for v in w]
    keep = 1.0 - c["drop"]
    reached = sum(1.0 - (1.0 - min(1.0, k * q) * keep) ** T for q in p)
    R = T * k * keep
    return dict(bytes=reached * _row_layout(H, I)["end"] + 4 * T * H + 8 * T * k, flops=6 * R * H * I)


# -------------------------------------------------------------------- exact
def _e4m3_64(v):
    """Nearest e4m3 value of each float64, ties to even, at most 448."""
    m, e = torch.frexp(v.abs())                     # v = m 2^e, m in [1/2, 1)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.sign(v) * (torch.round(v.abs() / step) * step).clamp_max(CODE_MAX)


def _rows_64(x):
    """Codes and scales of each 128 values of x [T, K] in 64 bits."""
    T, K = x.shape
    q, s = torch.empty_like(x), torch.empty((T, cdiv(K, BLK)), dtype=torch.float64, device=x.device)
    for b in range(s.shape[1]):
        part = x[:, b * BLK:(b + 1) * BLK]
        a = part.abs().max(dim=1).values.clamp_min(AMAX_MIN)
        s[:, b] = a / 448
        q[:, b * BLK:(b + 1) * BLK] = _e4m3_64(part * 448 / a[:, None])
    return q, s


def _spread(s, W):
    return torch.repeat_interleave(s, BLK, dim=1)[:, :W]


def _matrix_64(codes, s):
    """codes [N, K] bytes, s [ceil(N/128), ceil(K/128)] -> float64."""
    N, K = codes.shape
    w = codes.contiguous().view(torch.float8_e4m3fn).double()
    for b in range(s.shape[0]):
        w[b * BLK:(b + 1) * BLK] *= _spread(s[b:b + 1].double(), K)
    return w


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    T = c["T"]
    if c["op"] == "norm":
        def rms(v):
            return torch.sqrt(torch.square(v).sum(1, keepdim=True) / c["H"] + EPS)

        y = st["y"].double()
        v = y / rms(y) * (st["post"].double() + W_OFFSET)
        if c["gate"] != "none":
            a = st["gate"].double()
            a = a[:, None] if c["gate"] == "token" else a
            v = v * (a if c["gate"] == "channel" else 1 / (1 + torch.exp(-a)))
        r = st["residual"].double() + RESIDUAL_SCALE * v
        u = r / rms(r) * (st["pre"].double() + W_OFFSET)
        return [r, u, *_rows_64(u)] if c["quant"] else [r, u]
    if c["op"] == "quantize":
        x = st["x"].double()
        if c["act"] == "swiglu":
            x = x[:, : c["K"]] * torch.sigmoid(x[:, : c["K"]]) * x[:, c["K"]:]
        return list(_rows_64(x))
    if c["op"] == "gemm":
        x = st["xq"].contiguous().view(torch.float8_e4m3fn).double() * _spread(st["xs"].double(), c["K"])
        return x @ _matrix_64(st["wq"], st["ws"]).t()
    H, I = c["H"], c["I"]
    lay = _row_layout(H, I)
    hb, ib = lay["hb"], lay["ib"]
    q, s = _rows_64(st["x"].double())
    x = q * _spread(s, H)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in torch.unique(st["ids"]).tolist():
        if e < 0:
            continue
        t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        row = st["pool"][int(st["e2s"][e])]
        s13 = row[lay["s13"]:lay["s13"] + 8 * ib * hb].view(torch.float32).reshape(2 * ib, hb)
        gate = x[t] @ _matrix_64(row[: I * H].reshape(I, H), s13[:ib]).t()
        up = x[t] @ _matrix_64(row[I * H:lay["w2"]].reshape(I, H), s13[ib:]).t()
        q, s = _rows_64(gate * torch.sigmoid(gate) * up)
        s2 = row[lay["s2"]:lay["s2"] + 4 * hb * ib].view(torch.float32).reshape(hb, ib)
        y = (q * _spread(s, I)) @ _matrix_64(row[lay["w2"]:lay["s13"]].reshape(H, I), s2).t()
        out.index_add_(0, t, y * st["weights"][t, j].double()[:, None])
    return out
