"""The operators of a tuning step, as cases to measure.

linear_cross_entropy  softmax cross entropy of an output head (a solved layer, or a matrix), in pieces of the
                      vocabulary and without keeping the logits, with its gradients
adamw                 one AdamW step over many tensors at once, moments in 32 or in 8 bits, with the gradients'
                      global norm

`run` computes them in elementary torch operations, or with `own` through the package.
"""
import functools
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
LEVELS = {"s3": 8, "s4": 16, "s6": 64}   # scalar grids
E8_K = 65536
E8_RMS = 1.0660715                       # of the table's entries


def listed():
    def head(name, t, vocab, n, book, dtype, group=0, bias=False, padded=False, dx=True, dhead=True):
        return dict(name=name, op="cross_entropy", t=t, vocab=vocab, n=n, book=book, dtype=dtype, group=group,
                    bias=bias, padded=padded, dx=dx, dhead=dhead)

    def step(name, tensors, size, odd, dtype, bits, clip, decay):
        return dict(name=name, op="adamw", tensors=tensors, size=size, odd=odd, dtype=dtype, bits=bits, clip=clip,
                    decay=decay)
    return [
        # the smallest call: one token through a small 3-bit head, every gradient; latency alone
        head("ce_small", 1, 1000, 256, "s3", "fp32", bias=True),
        # one decoded token scored by a 2-bit head (the loss alone)
        head("ce_token_e8", 1, 32000, 4096, "e8", "bf16", dx=False, dhead=False),
        # perplexity of a text through a 2-bit head over a large vocabulary
        head("ce_text_e8", 2048, 128256, 4096, "e8", "bf16", padded=True, dx=False, dhead=False),
        # tuning the row scales of that head, and what lies below it, on a batch: the most work
        head("ce_tune_e8", 2048, 128256, 4096, "e8", "bf16"),
        # a short ragged batch, an odd vocabulary, a 4-bit head with groups of 128, a bias, padded positions
        head("ce_tune_g128", 509, 50257, 2048, "s4", "fp16", group=128, bias=True, padded=True),
        # the layers below an unquantized head are tuned: the gradient of its input alone
        head("ce_dense_dx", 777, 32000, 4096, "dense", "bf16", dhead=False),
        # an unquantized float32 head is tuned itself, on calibration activations
        head("ce_dense_fp32", 333, 32000, 1024, "dense", "fp32", bias=True),
        # the scale and the offset of one solved layer: the smallest step, latency alone
        step("adamw_layer", 2, 4096, False, "fp32", 32, False, 0.0),
        # scales and offsets by row of every layer of a model, their common norm clipped
        step("adamw_rows", 448, 8192, True, "fp32", 32, True, 0.0),
        # scales and offsets by groups of 128 of the layers of a model, moments in 8 bits
        step("adamw_groups8", 112, 229376, True, "fp32", 8, True, 0.01),
        # an unquantized bfloat16 head and its norms, moments in 8 bits, clipped
        step("adamw_head8", 3, 25000000, True, "bf16", 8, True, 0.1),
        # the same in float16 with 32-bit moments
        step("adamw_head32", 2, 12000000, True, "fp16", 32, False, 0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if rng.random() < 0.6:
        book = rng.choice(["e8", "e8", "s3", "s4", "s6", "dense", "dense"])
        t, vocab, n = _log_int(rng, 1, 2048), _log_int(rng, 500, 128256), _log_int(rng, 64, 4096)
        if book == "e8":
            n = max(8, n // 8 * 8)
        elif rng.random() < 0.7:
            n = n // 128 * 128 or 128
        group = rng.choice([0, 0, 128, 64]) if book[0] == "s" else 0
        dx, dhead = rng.choice([(True, True), (True, True), (True, False), (False, False)])
        # float32 operands and the gradients of groups and matrices are several products each
        costly = dtype == "fp32" or (dhead and (group or book == "dense"))
        t = max(1, min(t, 2048 * 128256 * 4096 // ((4 if costly else 1) * vocab * n)))
        return dict(op="cross_entropy", t=t, vocab=vocab, n=n, book=book, dtype=dtype, group=group if group < n else 0,
                    bias=rng.random() < 0.5, padded=rng.random() < 0.5, dx=dx, dhead=dhead)
    tensors = _log_int(rng, 1, 500)
    size = _log_int(rng, 100, 50000000 // tensors)
    return dict(op="adamw", tensors=tensors, size=size, odd=rng.random() < 0.7,
                dtype=dtype if rng.random() < 0.5 else "fp32", bits=rng.choice([8, 8, 32]), clip=rng.random() < 0.5,
                decay=rng.choice([0.0, 0.01, 0.1]))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


@functools.lru_cache(maxsize=1)
def _e8_table():
    """The first 65536 points of E8 in (squared norm, coordinates) order, and their cumulated shares of the codes."""
    pts = []
    for step in (0.0, 0.5):
        axis = np.arange(-3, 4) if step == 0.0 else np.arange(-3, 3)
        half = np.stack(np.meshgrid(*[axis + step] * 4, indexing="ij"), -1).reshape(-1, 4).astype(np.float32)
        half = half[(half ** 2).sum(1) <= 12]
        norm = (half ** 2).sum(1)
        a, b = np.nonzero(norm[:, None] + norm[None, :] <= 12)
        p = np.concatenate([half[a], half[b]], 1)
        pts.append(p[p.sum(1) % 2 == 0])
    pts = np.concatenate(pts)
    order = np.lexsort(tuple(pts[:, j] for j in range(7, -1, -1)) + ((pts ** 2).sum(1),))
    pts = np.ascontiguousarray(pts[order][:E8_K])
    # how often Gaussian weights of the table's rms meet each codeword, by their density, summed up
    share = np.exp(-(pts.astype(np.float64) ** 2).sum(1) / (2 * E8_RMS ** 2)).cumsum()
    return pts, (share / share[-1])


def _codes(case, g):
    """Codes, base codebook, scales and offsets of a solved head of Gaussian weights: logits of some three about zero."""
    m, n, group = case["vocab"], case["n"], case["group"]
    size = 2.5 / math.sqrt(n)
    if case["book"] == "e8":
        E, share = (torch.from_numpy(v).cuda() for v in _e8_table())
        u = torch.rand(m, n // 8, generator=g, device="cuda", dtype=torch.float64)
        codes = torch.searchsorted(share, u).clamp_max(E8_K - 1).int()
        return codes, E, (0.7 + 0.6 * _uniform(g, m)) * size / E8_RMS, None
    K = LEVELS[case["book"]]
    E = torch.arange(K, dtype=torch.float32, device="cuda").view(K, 1)
    width = group or n
    W = _normal(g, m, n) * size
    Wg = torch.nn.functional.pad(W, (0, -n % width), value=float("nan")).view(m, -1, width)
    lo = torch.nan_to_num(Wg, nan=float("inf")).amin(2)
    hi = torch.nan_to_num(Wg, nan=float("-inf")).amax(2)
    scale = ((hi - lo) / (K - 1)).clamp_min(1e-8)
    zero = torch.round(-lo / scale)
    codes = (torch.round(torch.nan_to_num(Wg) / scale[..., None]) + zero[..., None]).clamp(0, K - 1)
    codes = codes.view(m, -1)[:, :n].int().contiguous()
    offset = -scale * zero
    return codes, E, (scale if group else scale[:, 0].contiguous()), (offset if group else offset[:, 0].contiguous())


def _head_rows(s, rows):
    """Some of the head's rows, roughly (what a hidden state points at)."""
    if s["book"] == "dense":
        return s["W"][rows].float()
    w = s["E"][s["codes"][rows].long()].reshape(len(rows), s["n"])
    return w - w.mean(1, keepdim=True)


def _prepare_head(s, g):
    t, vocab, n, dt = s["t"], s["vocab"], s["n"], DTYPES[s["dtype"]]
    if s["book"] == "dense":
        s["W"] = (_normal(g, vocab, n) * (2.5 / math.sqrt(n)) * (0.7 + 0.6 * _uniform(g, vocab, 1))).to(dt)
    else:
        s["codes"], s["E"], s["scale"], s["offset"] = _codes(s, g)
    s["bias_v"] = 0.3 * _normal(g, vocab) if s["bias"] else None
    s["targets"] = torch.randint(vocab, (t,), generator=g, device="cuda").int()
    # states that see their next token coming, some clearly, some not at all; some channels are larger than others
    x = _normal(g, t, n) * torch.exp(0.3 * _normal(g, n))
    toward = _head_rows(s, s["targets"].long())
    toward = toward / toward.square().mean(1, keepdim=True).sqrt()
    x = x + toward * (2.0 / math.sqrt(n)) * _uniform(g, t, 1) * math.sqrt(math.log(vocab))
    s["x"] = x.to(dt)
    # a mean over the batch; float16 tuning scales its loss
    s["weights"] = torch.full((t,), (2.0 ** 10 if s["dtype"] == "fp16" else 1.0) / t, device="cuda")
    if s["padded"]:
        s["targets"][_uniform(g, t) < 0.2] = -1
    if own:
        import post_quantization_solver_amd as mpq
        s["head"] = s["W"] if s["book"] == "dense" else mpq.pack_layer(
            s["codes"], mpq.prepare_codebook(s["E"]), s["scale"], s["offset"], group=s["group"] or None)
    return s


LR, BETA1, BETA2, EPS, GRAD_SCALE, STEP = 1e-3, 0.9, 0.99, 1e-8, 2.0 ** -10, 40
BLOCK = 256                                 # moments of 8 bits: elements that share a scale


def _levels(fraction, dtype=torch.float64):
    """What codes of 7 (fraction = 3) or 8 bits (4) stand for, in units of the smallest."""
    half = 1 << fraction
    c = torch.arange(16 * half, device="cuda")
    e, f = c // half, c % half
    return torch.where(e == 0, f, (half + f) << (e - 1).clamp_min(0)).to(dtype)


def _tensor_sizes(s):
    """Sizes around `size`; odd ones do not fill their last block."""
    k = np.arange(s["tensors"])
    share = (0.25, 1.0, 0.5, 0.75)
    sizes = [max(1, int(s["size"] * share[i % 4])) if s["odd"] else s["size"] for i in k]
    return [v | 1 if s["odd"] and i % 3 == 2 else v for i, v in enumerate(sizes)]


def _prepare_step(s, g):
    dt = DTYPES[s["dtype"]]
    sizes = _tensor_sizes(s)
    places = [-(-v // BLOCK) * BLOCK for v in sizes]
    starts = [0] + list(np.cumsum(places))[:-1]
    total = sum(places)
    # parameters and moments of one tensor after another, each from a multiple of 256 on
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    kind = torch.zeros(total, device="cuda")
    scales = torch.exp(2.0 * _normal(g, len(sizes))).tolist()
    for at, v, k in zip(starts, sizes, scales):
        live[at:at + v] = True
        kind[at:at + v] = k
    s["at"] = live.nonzero()[:, 0]
    s["flat"] = torch.where(live, _normal(g, total), 0.0).to(dt)
    s["params"] = [s["flat"][at:at + v] for at, v in zip(starts, sizes)]
    # gradients of very different sizes, some rare; the moments of earlier ones like them
    size = kind * 1e-3 * torch.exp(_normal(g, total))
    grad = _normal(g, total) * size / GRAD_SCALE * (0.05 if s["dtype"] == "fp16" else 1.0)
    grad = torch.where(_uniform(g, total) < 0.05, 0.0, grad).to(dt)
    s["grads"] = [grad[at:at + v].clone() for at, v in zip(starts, sizes)]
    s["max_norm"] = float(0.5 * GRAD_SCALE * grad.double().square().sum().sqrt()) if s["clip"] else None
    s["step"] = torch.tensor([STEP], dtype=torch.int32, device="cuda")
    s["seed_v"] = int(torch.randint(1 << 31, (1,), generator=g, device="cuda"))
    m, r = 0.3 * _normal(g, total) * size, torch.sqrt(0.3 + _uniform(g, total)) * size
    if s["bits"] == 32:
        s["m"], s["v"] = torch.where(live, m, 0.0), torch.where(live, r * r, 0.0)
    else:
        (s["m"], s["m_scale"]), (s["r"], s["r_scale"]) = (
            _nearest(torch.where(live, v, 0.0), f) for v, f in ((m, 3), (r, 4)))
    if own:
        import post_quantization_solver_amd as mpq
        s["opt"] = mpq.AdamW(s["params"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=s["decay"],
                             state_bits=s["bits"], seed=s["seed_v"])
        s["opt"].load_state_dict({k: s[k] for k in ("step", "m", "v", "r", "m_scale", "r_scale") if k in s})
    return s


def _nearest(v, fraction):
    """8-bit codes of values and their blocks' scales, rounded to the nearest."""
    levels = _levels(fraction, torch.float32)
    b = v.view(-1, BLOCK)
    scale = b.abs().amax(1) / levels[-1]
    x = b.abs() / scale.clamp_min(1e-38)[:, None]
    code = torch.bucketize(x, (levels[1:] + levels[:-1]) / 2)
    if fraction == 3:
        code = code + 128 * ((b < 0) & (code > 0))
    return code.to(torch.uint8).view(-1), scale


def prepare(case, seed):
    g, s = _generator(seed), dict(case)
    return _prepare_head(s, g) if s["op"] == "cross_entropy" else _prepare_step(s, g)


# ------------------------------------------------------------------ the operators

def run(state):
    return _cross_entropy(state) if state["op"] == "cross_entropy" else _adamw(state)


def _entries(s):
    return s["E"][s["codes"].long()].reshape(s["vocab"], s["n"])


def _weights(s):
    """The head's weights in float32."""
    if s["book"] == "dense":
        return s["W"].float()
    w, a, o, n = _entries(s), s["scale"], s["offset"], s["n"]
    if s["group"]:
        a, o = (torch.repeat_interleave(v, s["group"], 1)[:, :n] for v in (a, o))
    else:
        a, o = a[:, None], (o[:, None] if o is not None else None)
    return a * w if o is None else a * w + o


def _cross_entropy(s):
    if own:
        import post_quantization_solver_amd as mpq
        r = mpq.linear_cross_entropy(s["x"], s["head"], s["targets"], bias=s["bias_v"], weights=s["weights"],
                                     need_dx=s["dx"], need_dhead=s["dhead"])
        if s["book"] != "dense" and s["offset"] is None:
            r.pop("doffset")
        return {k: v for k, v in r.items() if v is not None}
    x, W = s["x"].float(), _weights(s)
    z = x @ W.t()
    if s["bias_v"] is not None:
        z = z + s["bias_v"]
    tok = s["targets"].long()
    row, there = torch.arange(len(tok), device="cuda"), tok >= 0
    tok, weights = tok.clamp_min(0), torch.where(there, s["weights"], 0.0)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    own_mass = e[row, tok].double()
    total = e.sum(1, dtype=torch.float64)
    out = dict(loss=(weights.double() * (torch.log(total) - (z[row, tok] - top[:, 0]).double())).float())
    if not (s["dx"] or s["dhead"]):
        return out
    dz = e / total.float()[:, None]
    dz[row, tok] = ((own_mass - total) / total).float()
    dz = dz * weights[:, None]
    if s["dx"]:
        out["dx"] = (dz @ W).to(s["x"].dtype)
    if s["dhead"]:
        dW = dz.t() @ x
        if s["book"] == "dense":
            out["dweight"] = dW.to(s["x"].dtype)
        else:
            da = dW * _entries(s)
            if s["group"]:
                da, dW = (torch.nn.functional.pad(v, (0, -s["n"] % s["group"])).view(len(W), -1, s["group"]).sum(2)
                          for v in (da, dW))
            else:
                da, dW = da.sum(1), dW.sum(1)
            out["dscale"] = da
            if s["offset"] is not None:
                out["doffset"] = dW
        out["dbias"] = dz.sum(0)
    return out


def _mix(x):
    """A mixing of 32-bit words (in int64): shifts, and products with the fractions of the roots of 2 and 3."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xffffffff
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xffffffff
    return x ^ (x >> 16)


def _words(s, t, count):
    """Each position's random word of step t."""
    at = torch.arange(count, device="cuda")
    key = _mix(_mix(torch.tensor(s["seed_v"], device="cuda")) ^ t)
    return _mix((at & 0xffffffff) ^ _mix((key + (at >> 32)) & 0xffffffff))


def _stochastic(v, fraction, u):
    """8-bit codes of values (float64) and their blocks' scales, rounded up with the probability u says: of where the
    value (of a root: its square) lies between two codes'."""
    levels = _levels(fraction)
    b = v.view(-1, BLOCK)
    scale = (b.abs().amax(1) / levels[-1]).float()
    d = scale.double()[:, None]
    x = torch.where(d > 0, b.abs() / torch.where(d > 0, d, 1.0), 0.0).clamp_max(levels[-1].item())
    low = (torch.bucketize(x, levels, right=True) - 1).clamp_max(len(levels) - 2)
    power = 1 if fraction == 3 else 2
    below, above = levels[low] ** power, levels[low + 1] ** power
    code = low + (x ** power - below >= (1.0 - u.view(-1, BLOCK)) * (above - below))
    if fraction == 3:
        code = code + 128 * ((b < 0) & (code > 0))
    else:
        code = torch.where(b > 0, code.clamp_min(1), code)   # a root that is not zero stays so
    return code.to(torch.uint8).view(-1), scale


def _stood_for(code, scale, fraction):
    """The values of 8-bit codes, float64."""
    code = code.long()
    v = _levels(fraction)[code & 127 if fraction == 3 else code]
    v = v.view(-1, BLOCK) * scale.double()[:, None]
    return (torch.where(code.view(-1, BLOCK) > 127, -v, v) if fraction == 3 else v).view(-1)


def _round_param(p, dtype, u):
    """float32 values to the parameters' type; to 16 bits stochastically (u: 16 random bits)."""
    if dtype == torch.float32:
        return p
    drop = 16 if dtype == torch.bfloat16 else 13
    bits = p.contiguous().view(torch.int32)
    bits = (bits + (u & ((1 << drop) - 1)).int()) & -(1 << drop)
    return bits.view(torch.float32).to(dtype)


def _adamw(s):
    if own:
        opt = s["opt"]
        norm = opt.step(s["grads"], grad_scale=GRAD_SCALE, max_norm=s["max_norm"])
        m, v = opt.moments()
        out = dict(params=s["flat"], m=m, v=v)
        return dict(out, norm=norm) if s["clip"] else out
    small, flat, total = s["bits"] == 8, s["flat"], len(s["flat"])
    kind = torch.float64 if small else torch.float32
    g = torch.zeros(total, dtype=torch.float32, device="cuda")
    g[s["at"]] = torch.cat(s["grads"]).float()
    factor = torch.tensor(GRAD_SCALE, dtype=torch.float64, device="cuda")
    out = {}
    if s["clip"]:
        norm = g.double().square().sum().sqrt() * GRAD_SCALE
        factor = factor * (s["max_norm"] / norm).clamp_max(1.0)
        out["norm"] = norm.float()
    t = s["step"][0].long() + 1
    word = _words(s, t, total) if small or s["dtype"] != "fp32" else None
    g = g.to(kind) * factor.float().to(kind)
    if small:
        m, v = _stood_for(s["m"], s["m_scale"], 3), _stood_for(s["r"], s["r_scale"], 4) ** 2
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    live[s["at"]] = True
    c1, c2 = 1 / (1 - BETA1 ** t.double()), 1 / torch.sqrt(1 - BETA2 ** t.double())
    p = flat.float() * (1 - LR * s["decay"]) - (LR * (m * c1) / (v.sqrt() * c2 + EPS)).float()
    if small:
        s["m"], s["m_scale"] = _stochastic(m, 3, ((word & 0xffff) + 0.5) / 65536)
        s["r"], s["r_scale"] = _stochastic(v.sqrt(), 4, ((word >> 16) + 0.5) / 65536)
        m = _stood_for(s["m"], s["m_scale"], 3).float()
        v = (_stood_for(s["r"], s["r_scale"], 4) ** 2).float()
    else:
        s["m"], s["v"] = m, v
    if word is not None:
        word = _mix(word ^ 0x9E3779B9)
    flat.copy_(torch.where(live, _round_param(p, flat.dtype, word), flat))
    s["step"] = t.int().view(1)
    return dict(out, params=flat, m=m, v=v)


# ------------------------------------------------------------------ bounds and exact values

def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "adamw":
        count = float(sum(_tensor_sizes(case)))
        # 8 bits: the codes read and written, and the moments that they stand for
        moments = 2 * (1 + 1 + 4) + 16 / BLOCK if case["bits"] == 8 else 16
        return {"bytes": count * (3 * es + moments), "flops": 20.0 * count}
    t, vocab, n = case["t"], case["vocab"], case["n"]
    groups = -(-n // case["group"]) if case["group"] else 1
    dense, grads = case["book"] == "dense", case["dx"] or case["dhead"]
    if dense:
        head, dhead = es * vocab * n, es * vocab * n
    else:
        bits = 16 / 8 if case["book"] == "e8" else math.log2(LEVELS[case["book"]])
        dhead = 4 * vocab * groups * (1 if case["book"] == "e8" else 2)
        head = bits / 8 * vocab * n + dhead
    total = head + es * t * n * (2 if case["dx"] else 1) + 12 * t + 4 * vocab * case["bias"]
    if case["dhead"]:
        total += dhead + 4 * vocab
    # the logits; the input's gradient; a matrix's or the groups' gradient (a row's is a sum over its logits)
    products = 1 + (1 if case["dx"] else 0) + (1 if case["dhead"] and (dense or groups > 1) else 0)
    return {"bytes": total, "flops": 2.0 * products * t * vocab * n + (6.0 if grads else 4.0) * t * vocab}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_head(s) if s["op"] == "cross_entropy" else _exact_step(s)


def _exact_head(s):
    leaf = {}
    vocab, n = s["vocab"], s["n"]
    if s["book"] == "dense":
        W = leaf["dweight"] = s["W"].double().requires_grad_(s["dhead"])
    else:
        cols = torch.arange(n, device="cuda")
        d = s["E"].shape[1]
        e = torch.cat([s["E"].double()[c.long()[:, cols // d], cols % d] for c in s["codes"].split(8192)])
        group_of = cols // (s["group"] or n)
        leaf["dscale"] = s["scale"].double().requires_grad_(s["dhead"])
        W = leaf["dscale"].reshape(vocab, -1)[:, group_of] * e
        if s["offset"] is not None:
            leaf["doffset"] = s["offset"].double().requires_grad_(s["dhead"])
            W = W + leaf["doffset"].reshape(vocab, -1)[:, group_of]
    b = torch.zeros(vocab, dtype=torch.float64, device="cuda") if s["bias_v"] is None else s["bias_v"].double()
    leaf["dbias"] = b.requires_grad_(s["dhead"])
    x = leaf["dx"] = s["x"].double().requires_grad_(s["dx"])
    loss = torch.nn.functional.cross_entropy(torch.addmm(leaf["dbias"], x, W.t()), s["targets"].long(),
                                             ignore_index=-1, reduction="none") * s["weights"].double()
    wanted = [k for k, v in leaf.items() if v.requires_grad]
    out = dict(loss=loss.detach())
    if wanted:
        out.update(zip(wanted, torch.autograd.grad(loss.sum(), [leaf[k] for k in wanted])))
    return out


def _exact_step(s):
    """Tensor by tensor, in float64; parameters before they are rounded to their type."""
    t, blocks = STEP + 1, len(s["flat"]) // BLOCK
    grads = [g.double() * GRAD_SCALE for g in s["grads"]]
    out = {}
    if s["clip"]:
        norm = math.sqrt(sum(float((g * g).sum()) for g in grads))
        grads = [g * min(1.0, s["max_norm"] / norm) for g in grads]
        out["norm"] = torch.tensor(norm, dtype=torch.float64)
    def zeros():
        return torch.zeros(blocks * BLOCK, dtype=torch.float64, device="cuda")
    params, new_m, new_v, at = zeros(), zeros(), zeros(), 0
    key = _mix(_mix(torch.tensor(s["seed_v"])) ^ t).item()
    for p, g in zip(s["params"], grads):
        here, size = slice(at, at + len(p)), -(-len(p) // BLOCK) * BLOCK
        if s["bits"] == 8:
            def decode(name, bits):
                code = s[name][here].double()
                sign = torch.where(code >= 128, -1.0, 1.0) if bits == 3 else 1.0
                code = code % 128 if bits == 3 else code
                e = torch.floor(code / 2 ** bits)
                value = torch.where(e > 0, (2 ** bits + code % 2 ** bits) * torch.exp2(e - 1), code)
                scale = s[name + "_scale"].double().repeat_interleave(BLOCK)[here]
                return sign * value * scale
            m, v = decode("m", 3), decode("r", 4).square()
        else:
            m, v = s["m"][here].double(), s["v"][here].double()
        m, v = m + (1 - BETA1) * (g - m), v + (1 - BETA2) * (g.square() - v)
        denominator = (v / (1 - BETA2 ** t)).sqrt() + EPS
        params[here] = p.double() - LR * (s["decay"] * p.double() + m / (1 - BETA1 ** t) / denominator)
        if s["bits"] == 8:
            index = torch.arange(at, at + len(p), device="cuda")
            word = _mix((index % 2 ** 32) ^ _mix((index // 2 ** 32 + key) % 2 ** 32))
            def encode(v, bits, u):
                """Values rounded down, or up with the probability of where they (roots: their squares) lie between."""
                v = torch.nn.functional.pad(v, (0, size - len(p))).view(-1, BLOCK)
                u = torch.nn.functional.pad(u, (0, size - len(p))).view(-1, BLOCK)
                top = (2 ** (bits + 1) - 1) * 2.0 ** 14
                scale = (v.abs().amax(1, keepdim=True) / top).float().double()
                x = (v.abs() / torch.where(scale > 0, scale, 1.0)).clamp(0, top)
                gap = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** bits))) - bits)
                low = torch.floor(x / gap) * gap
                share = (x - low) / gap * (1.0 if bits == 3 else (x + low) / (2 * low + gap))
                x = low + gap * torch.floor(share + (u + 0.5) / 65536)
                if bits == 4:
                    x = torch.where(v > 0, x.clamp_min(1), x)
                return (torch.sign(v) * x.clamp_max(top) * scale).view(-1)[:len(p)]
            m, v = encode(m, 3, word % 65536), encode(v.sqrt(), 4, word // 65536).square()
        new_m[here], new_v[here] = m, v
        at += size
    return dict(out, params=params, m=new_m, v=new_v)
