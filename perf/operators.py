"""The operators on a solved layer and on a model's logits, as cases to measure.

linear            y = act(x W^T + bias) + residual of a quantized layer (codes, codebook, row or group affine)
linear_backward   its gradients: the input, the affine's scale and offset, the bias (the codes stay)
token_logprobs    log probability of given tokens, entropy and top alternatives of rows of logits
distill           KL divergence from a teacher's top log probabilities, with its gradient

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
    def linear(name, t, m, n, book, dtype, group=0, act="none", bias=False, residual=False, op="linear"):
        return dict(name=name, op=op, t=t, m=m, n=n, book=book, dtype=dtype, group=group, act=act, bias=bias,
                    residual=residual)
    return [
        # the smallest call: one token through a 64 x 256 3-bit layer; latency alone
        linear("linear_small", 1, 64, 256, "s3", "fp32", bias=True),
        # one decoded token through the 2-bit 4096 x 14336 down projection, residual added
        linear("linear_decode_e8", 1, 4096, 14336, "e8", "bf16", residual=True),
        # a batch of decoding sequences through a 4-bit layer with groups of 128, fp16 and a fused GELU
        linear("linear_decode_g128", 13, 2048, 8192, "s4", "fp16", group=128, act="gelu_tanh", bias=True),
        # a short chunk of a prompt through the square 2-bit layer
        linear("linear_chunk_e8", 65, 4096, 4096, "e8", "bf16", act="silu"),
        # a prompt (or a batch of calibration tokens) through the largest layer: the most work
        linear("linear_prefill_e8", 2048, 4096, 14336, "e8", "bf16", residual=True),
        # calibration activations as the front end holds them: float32, a ragged count of tokens
        linear("linear_calib_s3", 777, 2048, 2048, "s3", "fp32", bias=True),
        # tuning the group affine of a 4-bit layer under a fused activation
        linear("backward_g128", 1024, 2048, 8192, "s4", "bf16", group=128, act="gelu_tanh", bias=True,
               op="linear_backward"),
        # tuning the row scales of the square 2-bit layer on a short ragged batch
        linear("backward_e8", 333, 4096, 4096, "e8", "bf16", op="linear_backward"),
        # one decoded token's log probability and 20 alternatives; latency counts
        dict(name="logprobs_token", op="token_logprobs", t=1, vocab=32000, dtype="bf16", top=20, padded=False),
        # scoring a text: every position's token, entropy, and the 64 alternatives a student is tuned to
        dict(name="logprobs_text", op="token_logprobs", t=2048, vocab=128256, dtype="bf16", top=64, padded=False),
        # a small float32 tuning batch, tempered, an odd vocabulary, some padded positions
        dict(name="distill_odd", op="distill", t=509, vocab=50257, dtype="fp32", top=100, temperature=2.0, tail=False,
             padded=True),
        # a tuning batch of whole texts against the teacher's 64 log probabilities and their remainder
        dict(name="distill_text", op="distill", t=2048, vocab=128256, dtype="bf16", top=64, temperature=1.0,
             tail=True, padded=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "token_logprobs", "distill"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("linear", "linear_backward"):
        book = rng.choice(["e8", "e8", "s3", "s4", "s6"])
        t = _log_int(rng, 1, 2048)
        m = _log_int(rng, 64, 8192)
        n = _log_int(rng, 64, 14336)
        if book == "e8":
            n = n // 8 * 8
        elif rng.random() < 0.7:
            n = n // 128 * 128 or 128
        most = 2048 * 4096 * 14336 // (2 if op == "linear_backward" else 1)
        t = max(1, min(t, most // (m * n)))
        group = rng.choice([0, 0, 128, 64]) if book != "e8" else 0
        return dict(op=op, t=t, m=m, n=n, book=book, dtype=dtype, group=group if group < n else 0,
                    act=rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.5,
                    residual=op == "linear" and rng.random() < 0.5)
    vocab = _log_int(rng, 1000, 160000)
    t = min(_log_int(rng, 1, 4096), 2048 * 128256 * 2 // (BYTES[dtype] * vocab))
    top = rng.choice([1, 5, 20, 64, 100, 128])
    padded = rng.random() < 0.5
    if op == "token_logprobs":
        return dict(op=op, t=t, vocab=vocab, dtype=dtype, top=rng.choice([0, top]), padded=padded)
    tail = rng.random() < 0.5
    return dict(op=op, t=t, vocab=vocab, dtype=dtype, top=top,
                temperature=1.0 if tail else rng.choice([1.0, 2.0, 4.0]), tail=tail, padded=padded)


# ------------------------------------------------------------------ inputs

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


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _layer(case, g):
    """Codes, base codebook, scales and offsets of a layer of Gaussian weights."""
    m, n, group = case["m"], case["n"], case["group"]
    if case["book"] == "e8":
        E, share = (torch.from_numpy(v).cuda() for v in _e8_table())
        u = torch.rand(m, n // 8, generator=g, device="cuda", dtype=torch.float64)
        codes = torch.searchsorted(share, u).clamp_max(E8_K - 1).int()
        scale = (0.7 + 0.6 * torch.rand(m, generator=g, device="cuda")) / (E8_RMS * math.sqrt(n))
        return codes, E, scale, None
    K = LEVELS[case["book"]]
    E = torch.arange(K, dtype=torch.float32, device="cuda").view(K, 1)
    width = group or n
    pad = -n % width
    W = _normal(g, m, n) / math.sqrt(n)
    Wg = torch.nn.functional.pad(W, (0, pad), value=float("nan")).view(m, -1, width)
    lo = torch.nan_to_num(Wg, nan=float("inf")).amin(2)
    hi = torch.nan_to_num(Wg, nan=float("-inf")).amax(2)
    scale = ((hi - lo) / (K - 1)).clamp_min(1e-8)
    zero = torch.round(-lo / scale)
    codes = (torch.round(torch.nan_to_num(Wg) / scale[..., None]) + zero[..., None]).clamp(0, K - 1)
    codes = codes.view(m, -1)[:, :n].int().contiguous()
    offset = -scale * zero
    return codes, E, (scale if group else scale[:, 0].contiguous()), (offset if group else offset[:, 0].contiguous())


def prepare(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    t = case["t"]
    if case["op"] in ("linear", "linear_backward"):
        m, n = case["m"], case["n"]
        s["codes"], s["E"], s["scale"], s["offset"] = _layer(case, g)
        # a few channels of an LLM's activations are much larger than the rest
        s["x"] = (_normal(g, t, n) * torch.exp(0.5 * _normal(g, n))).to(dt)
        s["bias_v"] = 0.1 * _normal(g, m) if case["bias"] else None
        s["residual_v"] = _normal(g, t, m).to(dt) if case["residual"] else None
        if case["op"] == "linear_backward":
            s["dy"] = (_normal(g, t, m) * 0.02).to(dt)
            s["pre"] = _normal(g, t, m).to(dt) if case["act"] != "none" else None
        if own:
            import post_quantization_solver_amd as mpq
            s["layer"] = mpq.pack_layer(s["codes"], mpq.prepare_codebook(s["E"]), s["scale"], s["offset"],
                                        group=case["group"] or None)
        return s
    vocab, k = case["vocab"], case["top"]
    # rows of different sharpness around a shared trend
    base = _normal(g, t, vocab) * (1.5 + 2.0 * torch.rand(t, 1, generator=g, device="cuda"))
    s["logits"] = (base + 0.3 * _normal(g, t, vocab)).to(dt)
    drop = (torch.rand(t, generator=g, device="cuda") < 0.2) if case["padded"] else None
    if case["op"] == "token_logprobs":
        best = base.argmax(1)
        other = torch.randint(vocab, (t,), generator=g, device="cuda")
        s["tokens"] = torch.where(torch.rand(t, generator=g, device="cuda") < 0.6, best, other).int()
        if drop is not None:
            s["tokens"][drop] = -1
        return s
    values, ids = torch.topk(base, k, dim=1)
    s["ids"] = ids.int()
    s["teacher"] = values - torch.logsumexp(base, 1, keepdim=True)
    # a mean over the batch; float16 tuning scales its loss
    s["weights"] = torch.full((t,), (2.0 ** 14 if case["dtype"] == "fp16" else 1.0) / t, device="cuda")
    if drop is not None:
        s["weights"][drop] = 0.0
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    return _OPS[state["op"]](state)


def _weights(s):
    """The layer's weights in float32."""
    m, n = s["m"], s["n"]
    w = s["E"][s["codes"].long()].reshape(m, n)
    a, o = s["scale"], s["offset"]
    if s["group"]:
        a, o = (torch.repeat_interleave(v, s["group"], 1)[:, :n] for v in (a, o))
    else:
        a, o = a[:, None], (o[:, None] if o is not None else None)
    return a * w if o is None else a * w + o


def _act(u, name):
    if name == "relu":
        return torch.clamp_min(u, 0)
    if name == "silu":
        return u * torch.sigmoid(u)
    if name == "gelu":
        return 0.5 * u * (1 + torch.erf(u / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
    return u


def _act_slope(u, name):
    if name == "relu":
        return (u > 0).to(u.dtype)
    if name == "silu":
        q = torch.sigmoid(u)
        return q * (1 + u * (1 - q))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(u / math.sqrt(2))) + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (u + 0.044715 * u ** 3))
    return 0.5 * (1 + th) + 0.5 * u * (1 - th * th) * c * (1 + 3 * 0.044715 * u * u)


def _linear(s):
    if own:
        import post_quantization_solver_amd as mpq
        return mpq.linear(s["x"], s["layer"], bias=s["bias_v"], activation=None if s["act"] == "none" else s["act"],
                          residual=s["residual_v"])
    u = s["x"].float() @ _weights(s).t()
    if s["bias_v"] is not None:
        u = u + s["bias_v"]
    y = _act(u, s["act"])
    if s["residual_v"] is not None:
        y = y + s["residual_v"].float()
    return y.to(s["x"].dtype)


def _linear_backward(s):
    if own:
        import post_quantization_solver_amd as mpq
        r = mpq.linear_backward(s["dy"], s["x"], s["layer"], pre=s["pre"],
                                activation=None if s["act"] == "none" else s["act"])
        return dict(dx=r["dx"], dscale=r["dscale"], doffset=r["doffset"], dbias=r["dbias"])
    m, n, x = s["m"], s["n"], s["x"].float()
    du = s["dy"].float()
    if s["act"] != "none":
        du = du * _act_slope(s["pre"].float(), s["act"])
    dx = (du @ _weights(s)).to(s["x"].dtype)
    dw = du.t() @ x
    da = dw * s["E"][s["codes"].long()].reshape(m, n)
    if s["group"]:
        pad = -n % s["group"]
        da, dw = (torch.nn.functional.pad(v, (0, pad)).view(m, -1, s["group"]).sum(2) for v in (da, dw))
    else:
        da, dw = da.sum(1), dw.sum(1)
    return dict(dx=dx, dscale=da, doffset=dw, dbias=du.sum(0))


def _order_keys(z):
    """int64 keys of float rows that order by value, equal values by lowest index first."""
    bits = z.view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
    return (bits << 20) - torch.arange(z.shape[1], device=z.device)


def _token_logprobs(s):
    if own:
        import post_quantization_solver_amd as mpq
        r = mpq.token_logprobs(s["logits"], s["tokens"], top=s["top"])
        return {k: r[k] for k in ("logprob", "entropy", "lse") + (("top_ids", "top_logprobs") if s["top"] else ())}
    z, tok = s["logits"].float(), s["tokens"].long()
    top = z.amax(1, keepdim=True)
    d = z - top
    e = torch.exp(d)
    total = e.sum(1, dtype=torch.float64)
    lse = top[:, 0].double() + torch.log(total)
    entropy = torch.log(total) - (e * d).sum(1, dtype=torch.float64) / total
    picked = torch.gather(z, 1, tok.clamp_min(0)[:, None])[:, 0].double() - lse
    out = dict(logprob=torch.where(tok < 0, 0.0, picked).float(), entropy=entropy.float(), lse=lse.float())
    if s["top"]:
        ids = torch.topk(_order_keys(z), s["top"], dim=1).indices
        out["top_ids"] = ids.int()
        out["top_logprobs"] = (torch.gather(z, 1, ids).double() - lse[:, None]).float()
    return out


def _distill(s):
    T, tail, w = s["temperature"], s["tail"], s["weights"]
    if own:
        import post_quantization_solver_amd as mpq
        r = mpq.distill(s["logits"], s["ids"], s["teacher"], temperature=T, tail=tail, weights=w)
        return dict(loss=r["loss"], grad=r["grad"])
    z, ids = s["logits"].float() / T, s["ids"].long()
    teacher = s["teacher"].double() / T
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    log_q = torch.gather(z, 1, ids).double() - top.double() - torch.log(total)
    log_p = teacher if tail else teacher - torch.logsumexp(teacher, 1, keepdim=True)
    p = torch.exp(log_p)
    loss = (p * (log_p - log_q)).sum(1)
    q = e / total.float()
    if tail:
        rest = torch.scatter(e, 1, ids, 0.0).sum(1, keepdim=True, dtype=torch.float64) / total
        p_rest = (1 - p.sum(1, keepdim=True)).clamp_min(0)
        loss = loss + (p_rest * (torch.log(p_rest.clamp_min(1e-300)) - torch.log(rest)))[:, 0]
        listed_q = torch.gather(q, 1, ids)
        grad = q * (1 - p_rest / rest).float()
        grad = torch.scatter(grad, 1, ids, listed_q - p.float())
    else:
        grad = torch.scatter_add(q, 1, ids, -p.float())
    grad = grad * (w / T)[:, None]
    return dict(loss=(loss * w.double()).float(), grad=grad.to(s["logits"].dtype))


_OPS = {"linear": _linear, "linear_backward": _linear_backward, "token_logprobs": _token_logprobs,
        "distill": _distill}


# ------------------------------------------------------------------ bounds and exact values

def work(case):
    t, es = case["t"], BYTES[case["dtype"]]
    if case["op"] in ("linear", "linear_backward"):
        m, n = case["m"], case["n"]
        bits = 16 / 8 if case["book"] == "e8" else math.log2(LEVELS[case["book"]])
        groups = -(-n // case["group"]) if case["group"] else 1
        affine = 4 * m * groups * (1 if case["book"] == "e8" else 2)
        layer = bits / 8 * m * n + affine
        if case["op"] == "linear":
            return {"bytes": layer + es * t * (n + m * (2 if case["residual"] else 1)) + 4 * m * case["bias"],
                    "flops": 2.0 * t * m * n}
        return {"bytes": layer + es * t * (2 * n + m * (1 if case["act"] == "none" else 2)) + 8 * m * groups + 4 * m,
                "flops": 4.0 * t * m * n}
    cells = t * case["vocab"]
    if case["op"] == "token_logprobs":
        return {"bytes": es * cells + t * (16 + 8 * case["top"]), "flops": 5.0 * cells}
    return {"bytes": 2.0 * es * cells + t * (8 + 8 * case["top"]), "flops": 6.0 * cells}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x, W = s["x"].double(), _exact_layer(s)[0]
        u = torch.matmul(x, W.T)
        if s["bias_v"] is not None:
            u += s["bias_v"].double()
        y = u if s["act"] == "none" else _exact_act(u, s["act"])
        return y if s["residual_v"] is None else y + s["residual_v"].double()
    if case["op"] == "linear_backward":
        W, e, group_of = _exact_layer(s)
        du = s["dy"].double()
        if s["act"] != "none":
            u = s["pre"].double().requires_grad_()
            du = du * torch.autograd.grad(_exact_act(u, s["act"]).sum(), u)[0]
        dW = torch.matmul(du.T.contiguous(), s["x"].double())
        G = int(group_of[-1]) + 1
        zero = torch.zeros(s["m"], G, dtype=torch.float64, device="cuda")
        da, do = zero.index_add(1, group_of, dW * e), zero.index_add(1, group_of, dW)
        return dict(dx=torch.matmul(du, W), dscale=da.reshape(s["scale"].shape), doffset=do.reshape(s["scale"].shape),
                    dbias=du.sum(0))
    if case["op"] == "token_logprobs":
        out = dict(logprob=[], entropy=[], lse=[], top_ids=[], top_logprobs=[])
        for z, tok in zip(s["logits"].split(256), s["tokens"].split(256)):
            z = z.double()
            lp = torch.log_softmax(z, 1)
            out["lse"].append(torch.logsumexp(z, 1))
            out["entropy"].append(-(lp.exp() * lp).sum(1))
            row = torch.arange(len(tok), device="cuda")
            out["logprob"].append(torch.where(tok >= 0, lp[row, tok.clamp_min(0).long()], 0.0))
            order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            out["top_ids"].append(order.int())
            out["top_logprobs"].append(lp[row[:, None], order])
        out = {k: torch.cat(v) for k, v in out.items()}
        return out if case["top"] else {k: out[k] for k in ("logprob", "entropy", "lse")}
    losses, grads = [], []
    for z, ids, teacher, w in zip(*(s[k].split(256) for k in ("logits", "ids", "teacher", "weights"))):
        z, T = z.double().requires_grad_(), case["temperature"]
        lq = torch.log_softmax(z / T, 1)
        listed = torch.zeros_like(lq, dtype=torch.bool).scatter_(1, ids.long(), True)
        lt = teacher.double() / T
        if case["tail"]:
            rest = 1 - lt.exp().sum(1)
            lt = torch.cat([lt, rest.log()[:, None]], 1)
            lq_rest = torch.logsumexp(lq.masked_fill(listed, -math.inf), 1)
            pairs = torch.cat([lq.gather(1, ids.long()), lq_rest[:, None]], 1)
        else:
            lt, pairs = torch.log_softmax(lt, 1), lq.gather(1, ids.long())
        loss = (lt.exp() * (lt - pairs)).sum(1) * w.double()
        grads.append(torch.autograd.grad(loss.sum(), z)[0])
        losses.append(loss.detach())
    return dict(loss=torch.cat(losses), grad=torch.cat(grads))


def _exact_layer(s):
    """Weights, base entries (m x n) and each column's group, in 64 bits."""
    cols = torch.arange(s["n"], device="cuda")
    d = s["E"].shape[1]
    e = s["E"].double()[s["codes"].long()[:, cols // d], cols % d]
    group_of = cols // (s["group"] or s["n"])
    a = s["scale"].double().reshape(s["m"], -1)[:, group_of]
    W = a * e
    if s["offset"] is not None:
        W = W + s["offset"].double().reshape(s["m"], -1)[:, group_of]
    return W, e, group_of


def _exact_act(u, name):
    F = torch.nn.functional
    return {"relu": F.relu, "silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name](u)
