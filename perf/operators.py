"""The elementwise gated linear recurrence (scan, decode step, backward) and its 8-bit
activation checkpoint: cases to measure, the operators in plain torch operations, and
their definition in 64 bits.

    h_t = alpha_t h_{t-1} + w_t x_t,     alpha_t = exp(lambda_t)

per channel, lambda_t <= 0 the log-gate: given (``raw`` false) or log sigmoid of a raw
projection (``raw`` true); w_t = 1, or 1 - alpha_t (``complement``).  Tensors are
[B, T, D]; with ``seqs`` > 0, B = 1 and the T rows hold that many packed sequences.

The checkpoint keeps lambda_t and z_t = h_{t-1} (``complement``: h_{t-1} - x_t), all that
the backward multiplies, as e4m3 codes with one power-of-two scale per token and block of
128 channels.
"""
import torch

own = False

BLOCK = 128


# ---------------------------------------------------------------------------- cases
def listed():
    base = dict(op="fwd", dtype="bf16", B=1, T=1, D=1, seqs=0, raw=True, complement=True)
    return [
        # the tail of a chunked prompt, where only latency counts
        dict(base, name="fwd_f32_short", dtype="f32", B=2, T=100, D=512, raw=False, complement=False),
        # one prompt of ordinary length
        dict(base, name="fwd_prompt", B=1, T=1000, D=2048),
        # a training batch: B 8 sequences at the width of 16 heads of 128
        dict(base, name="fwd_train", B=8, T=4096, D=2048),
        # long context, one sequence: the width of 32 heads of 128
        dict(base, name="fwd_long", B=1, T=65536, D=4096, raw=False, complement=False),
        # packed documents of ragged lengths (some empty) and a width that no vector divides
        dict(base, name="fwd_packed_f32", dtype="f32", T=20011, D=1001, seqs=41),
        # gradients of a short sequence
        dict(base, name="bwd_f32_short", op="bwd", dtype="f32", B=2, T=200, D=500, raw=False),
        # the training batch's backward, from the activations as they are
        dict(base, name="bwd_train", op="bwd", B=8, T=4096, D=2048),
        # long context's backward
        dict(base, name="bwd_long", op="bwd", B=1, T=65536, D=4096, raw=False, complement=False),
        # the training batch's backward, from the 8-bit checkpoint
        dict(base, name="bwd_ckpt_train", op="bwd_ckpt", B=8, T=4096, D=2048),
        # a packed training step: forward that writes the checkpoint, backward that reads it
        dict(base, name="step_ckpt_packed", op="fwd_bwd_ckpt", T=32767, D=1024, seqs=29),
        # decoding a few sequences: latency
        dict(base, name="decode_small", op="decode", B=8, D=2048),
        # decoding a full serving batch: the state's bytes
        dict(base, name="decode_large", op="decode", B=4096, D=4096),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(2.0 ** rng.uniform(_log2(lo), _log2(hi))))))

    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "bwd_ckpt", "fwd_bwd_ckpt", "decode"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=1, T=1, D=log(64, 4096), seqs=0,
                raw=rng.random() < 0.6, complement=rng.random() < 0.6)
    if rng.random() < 0.6:
        case["D"] += -case["D"] % 8  # model widths are multiples of a vector; the others are drawn too
    if op == "decode":
        case["B"] = log(1, 4096)
        return case
    most = (1 << 26) // case["D"]
    rows = log(32, min(most, 131072))
    if rng.random() < 0.35:
        case["T"], case["seqs"] = rows, log(1, max(1, rows // 8))
    else:
        case["B"] = log(1, min(16, rows))
        case["T"] = max(1, rows // case["B"])
    return case


def _log2(v):
    return v.bit_length() - 1 + (v / (1 << (v.bit_length() - 1)) - 1)


def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    n = case["B"] * case["T"] * case["D"]
    state = 4 * (case["seqs"] or case["B"]) * case["D"]
    ckpt = 2 * n + 2 * case["B"] * case["T"] * -(-case["D"] // BLOCK)
    op = case["op"]
    if op == "decode":
        return {"bytes": 3 * n * eb + 2 * state, "flops": 8 * n}
    fwd = 3 * n * eb + 2 * state
    grads = 3 * n * eb + 2 * state                       # grad_h in, grad_x and grad_g out, state gradients
    saved = (3 if case["complement"] else 2) * n * eb + state
    total = {"fwd": fwd, "bwd": grads + saved, "bwd_ckpt": grads + ckpt, "fwd_bwd_ckpt": fwd + grads + 2 * ckpt}[op]
    return {"bytes": total, "flops": {"fwd": 10, "bwd": 14, "bwd_ckpt": 12, "fwd_bwd_ckpt": 24}[op] * n}


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    """Gates with a memory of a few to a thousand tokens, another for each channel and moving with
    each token; inputs, states and upstream gradients of unit size; what the forward saved."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, T, D = case["B"], case["T"], case["D"]
    N = case["seqs"] or B

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    raw = normal(B, T, D).add_(torch.rand(D, generator=gen, device="cuda").mul_(6).add_(1))
    s = dict(case, x=normal(B, T, D).to(dtype), g=(raw if case["raw"] else _log_sigmoid(raw)).to(dtype),
             s0=normal(N, D), cu=None)
    del raw
    if case["seqs"]:
        cuts = torch.randint(0, T + 1, (N - 1,), generator=gen, device="cuda").sort().values
        ends = torch.tensor([0, T], device="cuda")
        s["cu"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    if case["op"] == "decode":
        s["x"], s["g"], s["new"] = s["x"][:, 0].contiguous(), s["g"][:, 0].contiguous(), torch.empty_like(s["s0"])
    if "bwd" in case["op"]:
        s["dh"], s["dsT"] = normal(B, T, D).to(dtype), normal(N, D).mul_(0.1)
    if case["op"] == "fwd_bwd_ckpt":
        s["ckpt"] = torch.empty(_ckpt_layout(B * T, D)[-1], dtype=torch.uint8, device="cuda")
    if case["op"] == "bwd":
        s["h"] = _forward(s)[0].to(dtype)
    if case["op"] == "bwd_ckpt":
        s["ckpt"] = _pack(*_saved(s, _forward(s)[0]))
    return s


# ----------------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    dtype = s["x"].dtype
    if s["op"] == "decode":
        alpha, beta, _ = _gate(s)
        new = alpha * s["s0"] + (beta * s["x"].float() if s["complement"] else s["x"].float())
        return [new.to(dtype), new]
    if s["op"] == "fwd":
        h, sT = _forward(s)
        return [h.to(dtype), sT]
    if s["op"] == "bwd":
        alpha, beta, _ = _gate(s)
        return _backward(s, alpha, beta, _z(s, s["h"].float()))
    if s["op"] == "bwd_ckpt":
        return _backward_from(s, s["ckpt"])
    h, sT = _forward(s)
    return [h.to(dtype), sT] + _backward_from(s, _pack(*_saved(s, h)))


def _run_own(s):
    from gated_delta_rule_67_b200 import kda_scan_backward, kda_scan_backward_ckpt, kda_scan_fwd, kda_scan_step
    from gated_delta_rule_67_b200.binding import (KDA_PREP_GATE_LOGSIGMOID, KDA_SCAN_INPUT_COMPLEMENT,
                                                  KDA_SCAN_INPUT_PLAIN)
    how = dict(prep=KDA_PREP_GATE_LOGSIGMOID if s["raw"] else 0,
               input_gate=KDA_SCAN_INPUT_COMPLEMENT if s["complement"] else KDA_SCAN_INPUT_PLAIN)
    if s["op"] == "decode":
        return [kda_scan_step(s["x"], s["g"], s["s0"], out_state=s["new"], **how), s["new"]]
    how["cu_seqlens"] = s["cu"]
    if s["op"] == "fwd":
        return list(kda_scan_fwd(s["x"], s["g"], s["s0"], **how))
    if s["op"] == "bwd":
        d = kda_scan_backward(s["x"], s["g"], s["h"], s["dh"], s["s0"], s["dsT"], **how)
        return [d["dx"], d["dg"], d["dS0"]]
    out = list(kda_scan_fwd(s["x"], s["g"], s["s0"], checkpoint=s["ckpt"], **how)) if s["op"] == "fwd_bwd_ckpt" else []
    d = kda_scan_backward_ckpt(s["ckpt"], s["dh"], s["dsT"], **how)
    return out + [d["dx"], d["dg"], d["dS0"]]


# ------------------------------------------------------------------ the plain forms
def _log_sigmoid(r):
    return r.clamp(max=0) - torch.log1p(torch.exp(-r.abs()))


def _gate(s):
    """alpha, 1 - alpha and log alpha in fp32."""
    g = s["g"].float()
    if s["raw"]:
        return 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g)), _log_sigmoid(g)
    return torch.exp(g), -torch.expm1(g), g


def _edges(s):
    """Of each row: the sequence, whether it is the sequence's first row and its last."""
    B, T = s["x"].shape[:2]
    t = torch.arange(T, device="cuda")
    if s["cu"] is None:
        return torch.arange(B, device="cuda")[:, None].expand(B, T), (t == 0).expand(B, T), (t == T - 1).expand(B, T)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq[None], (t == cu[seq])[None], (t == cu[seq + 1] - 1)[None]


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t by doubling, in place (h_{-1} = 0)."""
    d = 1
    while d < u.shape[1]:
        u[:, d:] += a[:, d:] * u[:, :-d]
        a[:, d:] = a[:, d:] * a[:, :-d]
        d *= 2
    return u


def _rows_to_states(s, mask, seq, rows, empty):
    """rows[mask] as [N, D] by sequence; sequences without rows keep ``empty``."""
    out = empty.clone()
    out[seq[mask]] = rows[mask]
    return out


def _forward(s):
    alpha, beta, _ = _gate(s)
    seq, first, last = _edges(s)
    u = s["x"].float()
    u = beta * u if s["complement"] else u.clone()
    u[first] += alpha[first] * s["s0"][seq[first]]
    alpha[first] = 0
    h = _scan(alpha, u)
    return h, _rows_to_states(s, last, seq, h, s["s0"])


def _z(s, h):
    """What d alpha_t multiplies: h_{t-1}, less x_t where the input is weighed by 1 - alpha."""
    seq, first, _ = _edges(s)
    z = torch.roll(h, 1, 1)
    z[first] = s["s0"][seq[first]]
    return z - s["x"].float() if s["complement"] else z


def _saved(s, h):
    return _gate(s)[2], _z(s, h)


def _backward(s, alpha, beta, z):
    seq, first, last = _edges(s)
    d = s["dh"].float().clone()
    d[last] += s["dsT"][seq[last]]
    a = torch.roll(alpha, -1, 1)
    a[last] = 0
    d = _scan(a.flip(1), d.flip(1)).flip(1)
    dg = alpha * d * z
    if s["raw"]:
        dg = dg * beta
    ds0 = _rows_to_states(s, first, seq, alpha * d, s["dsT"])
    dtype = s["x"].dtype
    return [(beta * d if s["complement"] else d).to(dtype), dg.to(dtype), ds0]


def _backward_from(s, ckpt):
    B, T, D = s["x"].shape
    lam, z = (v.view(B, T, D) for v in _unpack(ckpt, B * T, D))
    return _backward(s, torch.exp(lam), -torch.expm1(lam), z)


def _ckpt_layout(rows, D):
    """Byte offsets: lambda codes [rows][P], z codes [rows][P], lambda scales [K][rows], z scales [K][rows],
    and the size; P = D rounded up to 16, K blocks of 128 channels, each part from a multiple of 256."""
    def up(v):
        return -(-v // 256) * 256

    codes, scales = up(rows * (-(-D // 16) * 16)), up(rows * -(-D // BLOCK))
    return 0, codes, 2 * codes, 2 * codes + scales, 2 * (codes + scales)


def _pack(lam, z):
    """The checkpoint's bytes.  The scale is 2^k with the least k >= -126 for which the block's largest
    magnitude is at most 448 * 2^k, held as k + 127; the code is value / 2^k rounded to e4m3."""
    D = lam.shape[-1]
    rows, P, K = lam.numel() // D, -(-D // 16) * 16, -(-D // BLOCK)
    at = _ckpt_layout(rows, D)
    out = torch.zeros(at[-1], dtype=torch.uint8, device=lam.device)
    for i, v in enumerate((lam, z)):
        full = torch.nn.functional.pad(v.reshape(rows, D), (0, K * BLOCK - D)).view(rows, K, BLOCK)
        m, e = torch.frexp(full.abs().amax(-1))
        k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
        k = torch.where(m == 0, torch.full_like(k, -126), k)
        code = torch.ldexp(full, -k[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, K * BLOCK)
        out[at[i]:at[i] + rows * P].view(rows, P)[:, :D] = code[:, :D]
        out[at[2 + i]:at[2 + i] + rows * K].view(K, rows)[:] = (k + 127).to(torch.uint8).t()
    return out


def _unpack(ckpt, rows, D):
    P, K = -(-D // 16) * 16, -(-D // BLOCK)
    at = _ckpt_layout(rows, D)
    got = []
    for i in range(2):
        code = ckpt[at[i]:at[i] + rows * P].view(rows, P)[:, :D].view(torch.float8_e4m3fn).float()
        k = ckpt[at[2 + i]:at[2 + i] + rows * K].view(K, rows).t().int() - 127
        got.append(torch.ldexp(code, k.repeat_interleave(BLOCK, 1)[:, :D]))
    return got


# ------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    g, x = s["g"].double(), s["x"].double()
    lam = -torch.nn.functional.softplus(-g, threshold=60) if s["raw"] else g
    if s["op"] == "decode":
        new = lam.exp() * s["s0"].double() - (torch.expm1(lam) if s["complement"] else -1) * x
        return [new, new]
    B, T, D = x.shape
    if s["cu"] is None:
        starts = {0: None}
        spans = None
    else:
        cu = s["cu"].tolist()
        spans = [(a, b) for a, b in zip(cu[:-1], cu[1:])]
        starts = {a: i for i, (a, b) in enumerate(spans) if b > a}
    ends = {T - 1: None} if spans is None else {b - 1: i for i, (a, b) in enumerate(spans) if b > a}
    s0 = s["s0"].double()
    z = sT = h = None
    if s["op"] != "bwd_ckpt":
        alpha, u = lam.exp(), (-torch.expm1(lam) * x if s["complement"] else x)
        h, prev, sT, c = torch.empty_like(x), torch.empty_like(x), s0.clone(), None
        for t in range(T):
            if t in starts:
                c = s0 if starts[t] is None else s0[starts[t]][None]
            prev[:, t] = c
            c = torch.addcmul(u[:, t], alpha[:, t], c)
            h[:, t] = c
            if t in ends:
                sT[slice(None) if ends[t] is None else slice(ends[t], ends[t] + 1)] = c
        if s["op"] == "fwd":
            return [h, sT]
        if s["op"] == "bwd":  # the saved outputs are inputs here
            prev[:, 1:] = s["h"][:, :-1].double()
            for t, i in starts.items():
                prev[:, t] = s0 if i is None else s0[i]
        z = prev - x if s["complement"] else prev
    if s["op"] == "bwd_ckpt":
        lam, z = _exact_values(s["ckpt"], B, T, D)
    elif s["op"] == "fwd_bwd_ckpt":
        lam, z = _exact_rounded(lam), _exact_rounded(z)
    alpha, beta = lam.exp(), -torch.expm1(lam)
    dy, dsT = s["dh"].double(), s["dsT"].double()
    dx, dg, ds0, c = torch.empty_like(x), torch.empty_like(x), dsT.clone(), None
    for t in range(T - 1, -1, -1):
        if t in ends:
            c = dsT if ends[t] is None else dsT[ends[t]][None]
        d = dy[:, t] + c
        c = alpha[:, t] * d
        dx[:, t], dg[:, t] = d, c
        if t in starts:
            ds0[slice(None) if starts[t] is None else slice(starts[t], starts[t] + 1)] = c
    if s["complement"]:
        dx *= beta
    dg *= z * beta if s["raw"] else z
    return ([h, sT] if s["op"] == "fwd_bwd_ckpt" else []) + [dx, dg, ds0]


def _exact_rounded(v):
    """Each value as its e4m3 code stands for it: 4 significant bits, no finer than 2^-9 of the scale."""
    B, T, D = v.shape
    out = torch.empty_like(v)
    for c in range(0, D, BLOCK):
        b = v[..., c:c + BLOCK]
        top = b.abs().amax(-1, keepdim=True)
        scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(min=-126))
        q = b / scale
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        out[..., c:c + BLOCK] = torch.round(q / step) * step * scale
    return out


def _exact_values(ckpt, B, T, D):
    """The checkpoint's values by the bit fields of its codes."""
    rows, P, K = B * T, -(-D // 16) * 16, -(-D // BLOCK)
    at, got = _ckpt_layout(B * T, D), []
    for i in range(2):
        c = ckpt[at[i]:at[i] + rows * P].view(rows, P)[:, :D].long()
        e, m = (c >> 3) & 15, (c & 7).double()
        v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
        k = ckpt[at[2 + i]:at[2 + i] + rows * K].view(K, rows).t().double() - 127
        got.append((torch.where(c >= 128, -v, v) * torch.exp2(k.repeat_interleave(BLOCK, 1)[:, :D])).view(B, T, D))
    return got
