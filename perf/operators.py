"""Cases of the element-wise optimizer operators: AdamW over many tensors with
moments in 32 or in 8 bits, the moments' conversion, and gradient clipping.

``run`` computes them in plain torch, or calls the library where ``own`` is
set; ``exact`` gives the same outputs from the definitions in 64 bits.

A case is a list of tensors.  Every tensor is a view of one flat buffer for
each quantity, so that the plain form works on whole buffers; the library
gets the views.  ``layout`` "aligned" starts every tensor at a multiple of 256
elements, "packed" puts them back to back from an odd offset on (the views of
one flat parameter buffer).  8-bit codes start at a multiple of 256 elements.

The moments in 8 bits, for each block of 256 elements of a tensor:
  m = e4m3(code) * 2^(SM - 127),           SM = max(1, E(max |m|) - 7)
  v = code as e5m3 without sign * 2^(SV - 127),  SV = max(1, E(max v) - 15)
with E the exponent field of the largest finite fp32 magnitude of the block,
m to the nearest code, v to the nearest or (stochastic) up with the
probability of its distance, and v > 0 never below code 1.  A step takes them of
the fp32 moments rn(rn(b1 m) + rn((1 - b1) g)) and rn(rn(b2 v) + rn((1 - b2) rn(g g))).
"""
import math
import random

import torch

own = False

BLOCK = 256
BETA1, BETA2, EPS, LR, STEP = 0.9, 0.999, 1e-8, 3e-4, 1000
MAX_NORM = 1.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WIDTH = {"f32": 4, "bf16": 2, "f16": 2, "": 0}
M32, M64 = (1 << 32) - 1, (1 << 64) - 1

_contexts = {}


def _context():
    """The library's context of a program: one for the device."""
    if "ctx" not in _contexts:
        from matrix_aware_optimizers_muon_b200 import Context
        _contexts["ctx"] = Context()
    return _contexts["ctx"]


# ---------------------------------------------------------------- the cases


def _case(name, op, kind, a, b, c=0, *, w="f32", g="bf16", copy="", layout="aligned", rounding="stochastic",
          device_scalars=False, zero_rows=0.0):
    """kind "equal": a tensors of b elements; "layer": one layer's seven
    matrices with hidden a, key/value width b and feed-forward width c;
    "experts": a experts' three b x c matrices; "ragged": a tensors of 1 to b
    elements drawn from seed c; zero_rows: share of 256-blocks that have had
    no gradient yet (rows of tokens not seen)."""
    d = dict(op=op, kind=kind, a=a, b=b, c=c, w=w, g=g, copy=copy, layout=layout, rounding=rounding,
             device_scalars=device_scalars, zero_rows=zero_rows)
    return dict(d, name=name) if name else d


def listed():
    return [
        # the norm weights of a 32-layer model, learning rate and step on the device: latency
        _case("adamw_norms", "adamw", "equal", 65, 4096, g="f32", device_scalars=True),
        # one layer of the dense model: fp32 master weights, bf16 gradients, bf16 copy for the next forward pass
        _case("adamw_layer", "adamw", "layer", 4096, 1024, 14336, copy="bf16"),
        # odd tensors back to back in a flat parameter buffer
        _case("adamw_ragged", "adamw", "ragged", 300, 200000, 7, g="f32", layout="packed"),
        # the same norm weights with 8-bit moments
        _case("adamw8_norms", "adamw8", "equal", 65, 4096, g="f32", rounding="nearest"),
        # sixteen experts of the mixture model, fp32 weights
        _case("adamw8_experts", "adamw8", "experts", 16, 768, 2048),
        # one layer of the dense model held in bf16 alone: the least bytes an element
        _case("adamw8_layer", "adamw8", "layer", 4096, 1024, 14336, w="bf16"),
        # odd tensors back to back, fp32 weights with an fp16 copy
        _case("adamw8_ragged", "adamw8", "ragged", 300, 200000, 7, g="f16", copy="f16", layout="packed"),
        # clipping small gradients on their way to an fp32 optimizer: latency
        _case("clip_norms", "clip", "equal", 65, 4096),
        # clipping a dense layer's bf16 gradients into the fp32 matrices that the Muon and SOAP steps take
        _case("clip_layer", "clip", "layer", 4096, 1024, 14336),
        # an embedding table's clipped step: the norm, then AdamW with its factor; most rows saw no token
        _case("clipped_embedding", "clipped", "equal", 1, 32000 * 4096, g="f32", zero_rows=0.75),
        # a checkpoint's fp32 moments into 8 bits and back
        _case("pack_ragged", "pack", "ragged", 300, 200000, 7, rounding="nearest"),
        _case("pack_experts", "pack", "experts", 16, 768, 2048),
    ]


def draw(rng):
    op = rng.choice(["adamw", "adamw", "adamw8", "adamw8", "adamw8", "clip", "clipped", "pack"])
    kind = rng.choice(["equal", "ragged", "layer", "experts"])
    if kind == "equal":
        a = int(2 ** rng.uniform(0, 8.5))
        b = max(1, int(2 ** rng.uniform(4, 26) / a) + rng.randrange(5))
        c = 0
    elif kind == "ragged":
        a, b, c = rng.randrange(2, 700), int(2 ** rng.uniform(6, 18.5)), rng.randrange(1 << 20)
    elif kind == "layer":
        a = 8 * rng.randrange(16, 250) + rng.choice([0, 0, 1, 5])
        b, c = max(1, a // rng.choice([1, 2, 4, 8])), a * rng.choice([2, 3, 4]) + rng.choice([0, 0, 3])
    else:
        a, b, c = rng.randrange(1, 17), rng.randrange(65, 900), rng.randrange(200, 2100)
    w = rng.choice(["f32", "f32", "bf16"])
    return _case(None, op, kind, a, b, c, w="f32" if op in ("clip", "pack") else w,
                 g=rng.choice(["f32", "bf16", "f16"]),
                 copy=rng.choice(["", "", "bf16", "f16"]) if w == "f32" and op not in ("clip", "pack") else "",
                 layout=rng.choice(["aligned", "packed"]), rounding=rng.choice(["nearest", "stochastic"]),
                 device_scalars=rng.random() < 0.3, zero_rows=rng.choice([0.0, 0.0, 0.5]))


def sizes_of(case):
    a, b, c = case["a"], case["b"], case["c"]
    if case["kind"] == "equal":
        return [b] * a
    if case["kind"] == "layer":
        return [a * a, b * a, b * a, a * a, c * a, c * a, a * c]
    if case["kind"] == "experts":
        return [b * c] * (3 * a)
    rng = random.Random(c)
    return [max(1, min(b, int(2 ** rng.uniform(0, math.log2(b))))) for _ in range(a)]


def work(case):
    n = sum(sizes_of(case))
    w, g, copy = WIDTH[case["w"]], WIDTH[case["g"]], WIDTH[case["copy"]]
    blocks = sum(-(-s // BLOCK) for s in sizes_of(case))
    step = {"bytes": n * (2 * w + g + copy + 16), "flops": 14 * n}
    if case["op"] in ("adamw", "clipped"):
        return step if case["op"] == "adamw" else {"bytes": step["bytes"], "flops": 17 * n}
    if case["op"] == "adamw8":  # codes and scales read and written, and the values they stand for (bf16) returned
        return {"bytes": n * (2 * w + g + copy + 4 + 4) + 4 * blocks, "flops": 18 * n}
    if case["op"] == "clip":
        return {"bytes": n * (g + 4), "flops": 3 * n}
    return {"bytes": n * (8 + 2 + 4) + 2 * blocks, "flops": 4 * n}


# ---------------------------------------------------------------- inputs


def _round_up(x, k):
    return -(-x // k) * k


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    sizes = sizes_of(case)
    packed = case["layout"] == "packed"
    starts, codes, at, cat = [], [], 1 if packed else 0, 0
    for s in sizes:
        starts.append(at)
        codes.append(cat)
        at += s if packed else _round_up(s, BLOCK)
        cat += _round_up(s, BLOCK)
    total, sum_ = at, sum(sizes)
    size = torch.tensor(sizes, device="cuda")
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), size) if total != sum_ or len(sizes) > 1 \
        else None

    def positions(first, all_):
        """Place of each element of the list in a flat buffer of all_ elements; None where it is its own number."""
        if all_ == sum_:
            return None
        ends = torch.cumsum(size, 0)
        shift = torch.tensor(first, device="cuda") - (ends - size)
        return torch.arange(sum_, device="cuda") + torch.repeat_interleave(shift, size)

    st = dict(case=dict(case), sizes=size, at=positions(starts, total), code_at=positions(codes, cat), elements=sum_,
              seed=12345)
    first = torch.tensor(codes, device="cuda")
    st["code_start"] = first
    dev = dict(device="cuda", generator=gen)
    # gradient scales differ from tensor to tensor, log-normally, around 1e-3
    std = 1e-3 * torch.exp(torch.randn(len(sizes), **dev))
    scale = torch.full((total,), 1e-3, device="cuda")
    one = std[tensor] if tensor is not None else std[0].expand(sum_)
    if st["at"] is None:
        scale = one.contiguous()
    else:
        scale[st["at"]] = one
    if case["zero_rows"]:
        seen = (torch.rand(-(-total // BLOCK), **dev) >= case["zero_rows"]).repeat_interleave(BLOCK)[:total]
    else:
        seen = None

    def normal():
        return torch.randn(total, **dev)

    G = normal().mul_(scale)
    M = normal().mul_(scale).mul_(0.23)
    V = torch.rand(total, **dev).add_(0.25).mul_(scale).mul_(scale)
    if seen is not None:
        G, M, V = G * seen, M * seen, V * seen
    st["G"] = G.to(TYPES[case["g"]])
    if case["op"] != "clip":
        st["W"] = normal().mul_(0.02).to(TYPES[case["w"]])
        st["copy"] = st["W"].to(TYPES[case["copy"]]) if case["copy"] else None
        # embeddings, norms and biases are left without decay: every third tensor
        st["decays"] = [0.0 if i % 3 == 0 else 0.1 for i in range(len(sizes))]
        st["M"], st["V"] = M, V
        st["lr"], st["step"] = LR, STEP
        if case["device_scalars"]:
            st["lr"] = torch.tensor(LR, device="cuda", dtype=torch.float32)
            st["step"] = torch.tensor(STEP, device="cuda", dtype=torch.int64)
    else:
        st["out"] = torch.zeros(total, device="cuda")
    if case["op"] in ("adamw8", "pack"):
        u8 = dict(device="cuda", dtype=torch.uint8)
        for k, n in (("M8", cat), ("V8", cat), ("MS", cat // BLOCK), ("VS", cat // BLOCK)):
            st[k] = torch.zeros(n, **u8)
        if case["op"] == "adamw8":
            _store(st, _take(M, st["at"]), _take(V, st["at"]), False)
            st["M"] = st["V"] = None
            st["M"] = torch.zeros(total, device="cuda", dtype=torch.bfloat16)  # what the codes stand for
            st["V"] = torch.zeros(total, device="cuda", dtype=torch.bfloat16)
        else:
            st["W"] = st["G"] = None
            st["MB"] = torch.zeros(total, device="cuda", dtype=torch.bfloat16)
            st["VB"] = torch.zeros(total, device="cuda", dtype=torch.bfloat16)
    if own:
        _handles(st, starts, codes, sizes)
    return st


def _handles(st, starts, codes, sizes):
    """The prepared tensor lists that a program keeps beside its parameters."""
    ctx, op = _context(), st["case"]["op"]

    def views(name, first=starts):
        t = st.get(name)
        return [None if t is None else t[a:a + s] for a, s in zip(first, sizes)]

    def scales(name):
        return [st[name][a // BLOCK:a // BLOCK + -(-s // BLOCK)] for a, s in zip(codes, sizes)]

    if op in ("clip", "clipped"):
        st["grads"] = ctx.clip_tensors([dict(G=g, out=o) for g, o in zip(views("G"), views("out"))]
                                       if op == "clip" else views("G"))
    if op in ("adamw", "clipped"):
        st["list"] = ctx.adamw_tensors([
            dict(W=w, G=g, M=m, V=v, copy=c, weight_decay=d) for w, g, m, v, c, d in
            zip(views("W"), views("G"), views("M"), views("V"), views("copy"), st["decays"])])
    if op in ("adamw8", "pack"):
        names = ("M", "V") if op == "adamw8" else ("MB", "VB")
        codes_ = dict(M8=views("M8", codes), V8=views("V8", codes), MS=scales("MS"), VS=scales("VS"))
        each = [dict(zip(codes_, c)) for c in zip(*codes_.values())]
        st["full"] = ctx.adamw8_moments([dict(e, M=m, V=v) for e, m, v in zip(each, views(names[0]), views(names[1]))])
        if op == "pack":
            st["from"] = ctx.adamw8_moments([dict(e, M=m, V=v) for e, m, v in zip(each, views("M"), views("V"))])
        else:
            st["list"] = ctx.adamw8_tensors([
                dict(e, W=w, G=g, copy=c, weight_decay=d) for e, w, g, c, d in
                zip(each, views("W"), views("G"), views("copy"), st["decays"])])


# ---------------------------------------------------------------- the plain form


def _take(x, at):
    return x if at is None else x[at]


def _put(x, at, values):
    if at is None:
        x.copy_(values)
    else:
        x[at] = values.to(x.dtype)


def _keys(seed, step, tensors):
    """Two 32-bit keys of each tensor's noise, as int64, from the seed, the step and the tensor's place in the list."""
    k = torch.arange(tensors, device="cuda")
    z = k * _signed(0xBB67AE8584CAA73B) + _wrap(step, 0x9E3779B97F4A7C15) + _signed(seed)
    for _ in range(2):
        z = z ^ ((z >> 32) & M32)
        z = z * _signed(0x6A09E667F3BCC909)
    z = z ^ ((z >> 32) & M32)
    return z & M32, (z >> 32) & M32


def _signed(x):
    x &= M64
    return x - (1 << 64) if x >> 63 else x


def _wrap(step, c):
    return step * _signed(c) if isinstance(step, torch.Tensor) else _signed(step * c)


def _noise(st):
    """16 random bits for each element's second moment and 16 for its weight, both functions of (seed, step, tensor, element)."""
    size = st["sizes"]
    k1, k2 = (torch.repeat_interleave(k, size) for k in _keys(st["seed"], st["step"], size.numel()))
    ends = torch.cumsum(size, 0)
    i = torch.arange(st["elements"], device="cuda") - torch.repeat_interleave(ends - size, size)
    x = (i >> 1) ^ k1
    x = (x * 0x9E3779B9) & M32
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667 + k2) & M32
    x = x ^ (x >> 15)
    x = (x * 0x9E3779B9) & M32
    x = x ^ (x >> 16)
    y = ((x ^ k1) * 0x6A09E667 + k2) & M32
    y = y ^ (y >> 16)
    half = (i & 1) * 16
    return (x >> half) & 0xFFFF, (y >> half) & 0xFFFF


def _blocks(st, x):
    """x of the list's elements in rows of 256, the tensors' ends filled up with zeros."""
    full = torch.zeros(st["M8"].numel(), device="cuda", dtype=x.dtype)
    _put(full, st["code_at"], x)
    return full.view(-1, BLOCK)


def _exponent(x):
    """Exponent field of each row's largest finite magnitude."""
    big = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(1)
    return big.view(torch.int32) >> 23


def _power(e):
    """2^(e - 127) for a biased exponent e >= 1, as fp32."""
    return (e << 23).view(torch.float32)


def _store(st, m, v, stochastic, bits=None):
    """Quantises the list's moments into the state's codes and scales."""
    mb, vb = _blocks(st, m), _blocks(st, v)
    ms, vs = (_exponent(mb) - 7).clamp(min=1), (_exponent(vb) - 15).clamp(min=1)
    q = (mb * _power(254 - ms)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    x = (vb * _power(254 - vs)[:, None] * 2.0 ** -112).view(torch.int32)
    if stochastic:
        r = x + (_blocks(st, bits.to(torch.int32)) * 16 + 8)
    else:
        r = x + 0x7FFFF + ((x >> 20) & 1)
    c = torch.where(vb > 0, (r >> 20).clamp(min=1), torch.zeros_like(r))
    c = torch.where(torch.isfinite(vb), c, torch.full_like(c, 255))
    for name, t in (("M8", q), ("V8", c), ("MS", ms), ("VS", vs)):
        old, new = st[name], t.to(torch.uint8).view(-1)
        if t.dim() == 2 and st["code_at"] is not None:  # the filling behind a tensor's end is not the state's
            old[st["code_at"]] = new[st["code_at"]]
        else:
            old.copy_(new)


def _load(st):
    """The moments that the state's codes stand for, of the list's elements, in fp32."""
    ms, vs = (_power(st[k].to(torch.int32)) for k in ("MS", "VS"))
    m = st["M8"].view(torch.float8_e4m3fn).float().view(-1, BLOCK) * ms[:, None]
    c = st["V8"].to(torch.int32).view(-1, BLOCK)
    v = (c << 20).view(torch.float32) * 2.0 ** 112 * vs[:, None]
    v = torch.where(c == 255, torch.full_like(v, math.nan), v)
    return _take(m.view(-1), st["code_at"]), _take(v.view(-1), st["code_at"])


def _stochastic_bf16(x, bits):
    """x to one of its two bf16 neighbours, up with the probability of its distance."""
    return ((x.view(torch.int32) + bits.to(torch.int32)) & -65536).view(torch.float32).to(torch.bfloat16)


def _adamw(st, g, m, v, bits=None):
    """New moments in the fixed order of roundings, and the weights written."""
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    lr, t = st["lr"], st["step"]
    if isinstance(t, torch.Tensor):
        c1, c2 = (1 - torch.pow(torch.tensor(b, dtype=torch.float64, device="cuda"), t) for b in (BETA1, BETA2))
        lr = lr.double()
        rate, root = (lr / c1).float(), (1 / c2.sqrt()).float()
    else:
        rate, root = lr / (1 - BETA1 ** t), 1 / math.sqrt(1 - BETA2 ** t)
    decay = torch.tensor(st["decays"], dtype=torch.float64, device="cuda")
    decay = torch.repeat_interleave((1 - lr * decay).float(), st["sizes"])
    w = _take(st["W"], st["at"]).float() * decay - (m * rate) / (v.sqrt() * root + EPS)
    if bits is not None and st["W"].dtype == torch.bfloat16:
        _put(st["W"], st["at"], _stochastic_bf16(w, bits))
    else:
        _put(st["W"], st["at"], w)
    if st["copy"] is not None:
        _put(st["copy"], st["at"], w.to(st["copy"].dtype))
    return m, v


def _norm(st):
    """The list's 2-norm (a long sum: in 64 bits) and the factor that brings it to MAX_NORM at most."""
    g = _take(st["G"], st["at"]).double()
    norm = (g * g).sum().sqrt()
    factor = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    return norm.float(), factor.float()


def _outputs(st):
    return {"W": st["W"], "M": st["M"], "V": st["V"], "copy": st["copy"]}


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    stochastic = case["rounding"] == "stochastic"
    if own:
        ctx = _context()
        seed = st["seed"] if stochastic else None
        hyper = dict(lr=st.get("lr"), beta1=BETA1, beta2=BETA2, eps=EPS)
        if op == "adamw":
            ctx.adamw_step(st["list"], st["step"], seed=seed, **hyper)
            return _outputs(st)
        if op == "adamw8":
            ctx.adamw8_step(st["list"], st["step"], seed=seed, **hyper)
            ctx.adamw8_unpack(st["full"])
            return _outputs(st)
        if op == "clip":
            norm, factor = ctx.clip_grads(st["grads"], MAX_NORM)
            return {"norm": norm, "factor": factor, "out": st["out"]}
        if op == "clipped":
            norm, factor = ctx.clip_grads(st["grads"], MAX_NORM, apply=False)
            ctx.adamw_step(st["list"], st["step"], seed=seed, grad_scale=factor, **hyper)
            return dict(_outputs(st), norm=norm)
        ctx.adamw8_pack(st["from"], seed=seed, step=st["step"])
        ctx.adamw8_unpack(st["full"])
        return {"M": st["MB"], "V": st["VB"]}
    at = st["at"]
    bits, wbits = _noise(st) if stochastic and (op in ("adamw8", "pack") or case["w"] == "bf16") else (None, None)
    if op == "clip":
        norm, factor = _norm(st)
        _put(st["out"], at, _take(st["G"], at).float() * factor)
        return {"norm": norm, "factor": factor, "out": st["out"]}
    if op in ("adamw", "clipped"):
        g = _take(st["G"], at).float()
        if op == "clipped":
            norm, factor = _norm(st)
            g = g * factor
        m, v = _adamw(st, g, _take(st["M"], at), _take(st["V"], at), wbits)
        _put(st["M"], at, m)
        _put(st["V"], at, v)
        return _outputs(st) if op == "adamw" else dict(_outputs(st), norm=norm)
    if op == "adamw8":
        m, v = _adamw(st, _take(st["G"], at).float(), *_load(st), wbits)
        _store(st, m, v, stochastic, bits)
        m, v = _load(st)
        _put(st["M"], at, m)
        _put(st["V"], at, v)
        return _outputs(st)
    _store(st, _take(st["M"], at), _take(st["V"], at), stochastic, bits)
    m, v = _load(st)
    _put(st["MB"], at, m)
    _put(st["VB"], at, v)
    return {"M": st["MB"], "V": st["VB"]}


# ---------------------------------------------------------------- 64 bits


def _grid(x, mantissa, least, up=None):
    """x (fp64) on the grid of floats with so many mantissa bits and the least exponent 2^least: nearest, ties to even,
    or up where its distance to the lower neighbour and `up` (both in steps) reach one."""
    e = (torch.frexp(x)[1] - 1).clamp(min=least)
    step = torch.ldexp(torch.ones_like(x), e - mantissa)
    return (torch.round(x / step) if up is None else torch.floor(x / step + up)) * step


def _block_max(st, x, first):
    """For each element the largest magnitude of its block (the blocks' numbers start at first / 256)."""
    ends = torch.cumsum(st["sizes"], 0)
    inside = torch.arange(st["elements"], device="cuda") - torch.repeat_interleave(ends - st["sizes"], st["sizes"])
    number = torch.repeat_interleave(first // BLOCK, st["sizes"]) + inside // BLOCK
    big = torch.zeros(int(number[-1]) + 1, dtype=x.dtype, device="cuda")
    big.scatter_reduce_(0, number, x.abs(), "amax")
    return big[number], inside


def _held(st, m, v, noise=None):
    """The values that moments (fp64) have once held in 8 bits."""
    bm, _ = _block_max(st, m, st["code_start"])
    e = torch.frexp(bm.clamp(min=2.0 ** -126))[1] - 1
    s = torch.ldexp(torch.ones_like(m), (e - 7).clamp(min=-126))
    hm = _grid(m.abs() / s, 3, -6) * s * torch.sign(m)
    bv, _ = _block_max(st, v, st["code_start"])
    e = torch.frexp(bv.clamp(min=2.0 ** -126))[1] - 1
    s = torch.ldexp(torch.ones_like(v), (e - 15).clamp(min=-126))
    up = None if noise is None else (noise.double() * 16 + 8) / 2 ** 20
    hv = torch.where(v > 0, _grid(v / s, 3, -14, up).clamp(min=2.0 ** -17) * s, torch.zeros_like(v))
    return hm, hv


def _codes64(st):
    """The values that the state's 8-bit codes stand for, by their fields."""
    at = torch.arange(st["M8"].numel(), device="cuda") if st["code_at"] is None else st["code_at"]
    c, d = st["M8"][at].long(), st["V8"][at].long()
    sm, sv = st["MS"][at // BLOCK].long() - 127, st["VS"][at // BLOCK].long() - 127
    f, e = c % 8, (c // 8) % 16
    one = torch.ones((), dtype=torch.float64, device="cuda")
    m = torch.where(e > 0, 8 + f, f).double() * torch.ldexp(one, e.clamp(min=1) - 10 + sm) * (1 - 2 * (c // 128))
    f, e = d % 8, d // 8
    return m, torch.where(e > 0, 8 + f, f).double() * torch.ldexp(one, e.clamp(min=1) - 18 + sv)


def _fp32_moments(st, g):
    """The new moments that the codes are taken of: by the definition fp32 values, each product and sum rounded once.
    The old codes and 16-bit gradients have so few bits that 0.9 m + 0.1 g is often a tie of two codes, which only
    a fixed order of roundings decides."""
    def r(x):
        return x.float().double()

    m, v = _codes64(st)
    b1, c1, b2, c2 = (r(torch.tensor(b, dtype=torch.float64)).item() for b in (BETA1, 1 - BETA1, BETA2, 1 - BETA2))
    return r(r(b1 * m) + r(c1 * g)), r(r(b2 * v) + r(c2 * r(g * g)))


def _mul64(a, b):
    """a * b mod 2^32 of values below 2^32, by halves."""
    return (a * (b & 0xFFFF) + (((a * (b >> 16)) & 0xFFFF) << 16)) & M32


def _bits64(st):
    """The noise bits by the definition, over Python integers for the keys."""
    keys, step = [], int(st["step"])
    for k in range(st["sizes"].numel()):
        z = (k * 0xBB67AE8584CAA73B + step * 0x9E3779B97F4A7C15 + st["seed"]) & M64
        for _ in range(2):
            z = ((z ^ (z >> 32)) * 0x6A09E667F3BCC909) & M64
        z ^= z >> 32
        keys.append((z & M32, z >> 32))
    k1, k2 = (torch.tensor(k, device="cuda").repeat_interleave(st["sizes"]) for k in zip(*keys))
    i = torch.cat([torch.arange(int(s), device="cuda") for s in st["sizes"].tolist()])
    x = _mul64((i // 2) ^ k1, 0x9E3779B9)
    x = (_mul64(x ^ (x >> 16), 0x6A09E667) + k2) & M32
    x = _mul64(x ^ (x >> 15), 0x9E3779B9)
    x = x ^ (x >> 16)
    y = (_mul64(x ^ k1, 0x6A09E667) + k2) & M32
    y = y ^ (y >> 16)
    odd = i % 2 == 1
    return torch.where(odd, x >> 16, x & 0xFFFF), torch.where(odd, y >> 16, y & 0xFFFF)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, at = case["op"], st["at"]
    stochastic = case["rounding"] == "stochastic"

    def laid(before, values):
        out = before.double()
        if at is None:
            return values
        out[at] = values
        return out

    def of(name):
        return _take(st[name], at).double()

    noise, wnoise = _bits64(st) if stochastic and (op in ("adamw8", "pack") or case["w"] == "bf16") else (None, None)
    if op == "pack":
        m, v = _held(st, of("M"), of("V"), noise)
        return {"M": laid(st["MB"], m), "V": laid(st["VB"], v)}
    g = of("G")
    norm = torch.linalg.vector_norm(g)
    factor = torch.clamp(MAX_NORM / (norm + 1e-6), max=1)
    if op == "clip":
        return {"norm": norm, "factor": factor, "out": laid(st["out"], g * factor)}
    m, v = _codes64(st) if op == "adamw8" else (of("M"), of("V"))
    if op == "clipped":
        g = g * factor
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    lr, t = float(st["lr"]), int(st["step"])
    decay = torch.tensor(st["decays"], dtype=torch.float64, device="cuda").repeat_interleave(st["sizes"])
    w = of("W")
    w = w - lr * decay * w - lr * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    copy = None if st["copy"] is None else laid(st["copy"], w)
    if st["W"].dtype == torch.bfloat16 and stochastic:
        w = _grid(w.abs(), 7, -126, wnoise.double() / 65536) * torch.sign(w)
    out = {"W": laid(st["W"], w), "copy": copy}
    if op == "adamw8":
        m, v = _held(st, *_fp32_moments(st, of("G")), noise)
    out.update(M=laid(st["M"], m), V=laid(st["V"], v))
    return dict(out, norm=norm) if op == "clipped" else out
