"""Cases of the serving and dropout operators of the QLoRA layer, their plain
torch forms and their 64-bit values.

Operators (a case's "op"):

  slots   token_slots            the adapter slot of every token, from request lengths
  multi   linear_fwd_slots       the layer with one low-rank adapter per request
  keep    dropout_keep_bits      keep mask of the counter-based LoRA dropout, as bits
  fwd     linear_fwd_dropout_rng the layer with that dropout, its mask never stored
  bwd     linear_bwd_dropout_rng its backward

`own` selects the framework's calls; otherwise run() computes the same values
with elementary torch operations in fp32.
"""

import math

import numpy as np
import torch

own = False

_M32 = 0xFFFFFFFF


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a small server: 48 requests of one token each
        dict(name="slots decode", op="slots", requests=48, tokens=48, decode=True),
        # packed prompts of a thousand requests, some of them empty, padded to a fixed token count
        dict(name="slots packed", op="slots", requests=1000, tokens=131072, decode=False),
        # one user decoding on a 7B attention projection: the smallest call of the layer
        dict(name="multi 7B one token", op="multi", M=1, n_in=4096, n_out=4096, r=16, n=8, requests=1),
        # sixteen users, each with an adapter of their own, on a 70B up projection
        dict(name="multi 70B up 16", op="multi", M=16, n_in=8192, n_out=28672, r=16, n=32, requests=16),
        # a full decode batch over many adapters on the 70B down projection
        dict(name="multi 70B down 128", op="multi", M=128, n_in=28672, n_out=8192, r=16, n=64, requests=128),
        # packed prompts of a few requests on a 65B gate projection, with padding at the end
        dict(name="multi 65B gate prompts", op="multi", M=2011, n_in=8192, n_out=22016, r=64, n=8, requests=9),
        # the mask of one 7B attention projection, drawn for inspection
        dict(name="keep 7B attention", op="keep", M=4096, n_in=4096, p=0.05),
        # the mask of a 7B down projection at the longest training batch
        dict(name="keep 7B down", op="keep", M=8192, n_in=11008, p=0.05),
        # a training step's forward and backward: 7B attention, 7B MLP and 65B gate
        dict(name="fwd 7B attention", op="fwd", M=4096, n_in=4096, n_out=4096, r=16, p=0.05),
        dict(name="fwd 7B up", op="fwd", M=8192, n_in=4096, n_out=11008, r=16, p=0.05),
        dict(name="bwd 7B attention", op="bwd", M=4096, n_in=4096, n_out=4096, r=16, p=0.05),
        dict(name="bwd 65B gate", op="bwd", M=2048, n_in=8192, n_out=22016, r=64, p=0.05),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["slots", "multi", "multi", "multi", "keep", "fwd", "bwd", "bwd"])
    if op == "slots":
        requests, decode = _log_int(rng, 1, 1000), rng.random() < 0.5
        return dict(op=op, requests=requests, decode=decode,
                    tokens=requests if decode else _log_int(rng, max(1, requests), 131072))
    n_in, n_out = (64 * _log_int(rng, 4, 172) for _ in range(2))
    M = _log_int(rng, 1, min(8192, 360000000000 // (n_in * n_out)))     # no more than the largest listed
    if op == "keep":
        return dict(op=op, M=M, n_in=n_in, p=round(rng.uniform(0.0, 0.5), 3))
    r = rng.choice([8, 16, 32, 64, _log_int(rng, 1, 96)])
    if op == "multi":
        requests = M if M <= 256 and rng.random() < 0.7 else _log_int(rng, 1, min(M, 64))
        return dict(op=op, M=M, n_in=n_in, n_out=n_out, r=r, n=_log_int(rng, 1, min(128, 2048 // r)),
                    requests=requests)
    return dict(op=op, M=M, n_in=n_in, n_out=n_out, r=r, p=round(rng.uniform(0.01, 0.3), 3))


# ------------------------------------------------------------------ inputs
def _levels():
    """The 16 NF4 levels: normal quantiles with an exact zero, ascending, fp32."""
    d = 1.0 - (1.0 / 32 + 1.0 / 30) / 2
    i8, i7 = torch.arange(8, dtype=torch.float64), torch.arange(7, dtype=torch.float64)
    top = torch.special.ndtri(torch.tensor(d, dtype=torch.float64))
    pos = torch.special.ndtri(d - i8 * (d - 0.5) / 8) / top
    neg = -torch.special.ndtri(d - i7 * (d - 0.5) / 7) / top
    return torch.cat([neg, torch.zeros(1, dtype=torch.float64), pos.flip(0)]).float()


def _weight(n_out, n_in, g, std):
    """A normal weight in the stored format: packed codes, 8-bit scale codes, steps, mean."""
    lev = _levels().cuda()
    mid = (lev[1:] + lev[:-1]) / 2
    W = torch.randn(n_out * n_in // 64, 64, generator=g, device="cuda") * std
    c = W.abs().amax(1)
    code = torch.searchsorted(mid, W / c[:, None], out_int32=True).to(torch.uint8)
    del W
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).reshape(n_out, n_in // 2).contiguous()
    mean = c.double().mean().float().reshape(1)
    dev = torch.zeros(-(-c.numel() // 256) * 256, device="cuda")
    dev[:c.numel()] = c - mean
    step = dev.view(-1, 256).abs().amax(1) / 127
    q8 = torch.where(step[:, None] > 0, dev.view(-1, 256) / step[:, None], 0).round().clamp(-127, 127)
    return dict(codes=codes, q8=q8.to(torch.int8).reshape(-1)[:c.numel()].contiguous(), step2=step.contiguous(),
                mean=mean)


def _bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


def _requests(case, g):
    """Request lengths and slots: one token each, or ragged with empty requests and unused tokens at the end."""
    n_req, tokens = case["requests"], case.get("tokens", case.get("M"))
    if n_req == tokens:
        lengths = torch.ones(n_req, dtype=torch.int64, device="cuda")
    else:
        share = torch.rand(n_req, generator=g, device="cuda") ** 2
        share = share * (torch.rand(n_req, generator=g, device="cuda") > 0.05)
        lengths = (share / share.sum().clamp(min=1e-6) * (0.97 * tokens)).long()
    n = case.get("n", 64)
    slots = torch.randint(0, n, (n_req,), generator=g, device="cuda")
    # now and then a request runs on the bare base model
    slots = torch.where(torch.rand(n_req, generator=g, device="cuda") < 0.05, torch.full_like(slots, -1), slots)
    if n_req == 1:
        slots.zero_()
    return lengths.int(), slots.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)
    s = dict(case)
    if s["op"] == "slots":
        s["lengths"], s["slots"] = _requests(case, g)
        return s
    if s["op"] in ("keep", "fwd", "bwd"):
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")
    if s["op"] == "keep":
        return s
    M, n_in, n_out, r = s["M"], s["n_in"], s["n_out"], s["r"]
    s["w"] = _weight(n_out, n_in, g, 0.02)
    s["x"] = _bf16(g, M, n_in)
    lead = (s["n"],) if s["op"] == "multi" else ()
    s["A"] = ((torch.rand(*lead, r, n_in, generator=g, device="cuda") * 2 - 1) / math.sqrt(n_in)).bfloat16()
    s["B"] = _bf16(g, *lead, n_out, r, std=0.01)
    if s["op"] == "multi":
        lengths, slots = _requests(case, g)
        s["ids"] = _slots_plain(lengths, slots, M)
        s["scale"] = torch.rand(s["n"], generator=g, device="cuda") * 2 + 0.5
    else:
        s["alpha"] = 2.0 * r
    if s["op"] == "bwd":
        s["dh"] = _bf16(g, M, n_out)
        s["us"] = _us_plain(s).bfloat16()          # what the forward handed on
    return s


# ------------------------------------------------------------ plain forms
def _slots_plain(lengths, slots, tokens):
    end = torch.cumsum(lengths.clamp(min=0).long(), 0)
    t = torch.arange(tokens, device=end.device)
    k = torch.searchsorted(end, t, right=True)
    return torch.where(k < end.numel(), slots[k.clamp(max=end.numel() - 1)], -1).int()


def _dequant_plain(w):
    """bf16(level * scale) of every weight, in fp32."""
    lev = _levels().to(w["codes"].device)
    code = torch.stack([w["codes"] & 15, w["codes"] >> 4], -1).reshape(-1, 64).int()
    q8 = w["q8"].float()
    step = w["step2"].repeat_interleave(256)[:q8.numel()]
    c = q8 * step + w["mean"]
    return (lev[code] * c[:, None]).bfloat16().float().reshape(w["codes"].shape[0], -1)


def _threshold(p):
    """The dropped share of 65536 and the share kept."""
    t = min(65535, int(round(p * 65536)))
    return t, 1.0 - t / 65536


def _keep_plain(rng, p, M, n):
    """Keep mask [M, n]: Philox4x32 with 7 rounds (Salmon et al., "Parallel
    random numbers: as easy as 1, 2, 3", 2011), key = seed, counter =
    (column / 8, row, offset); each 16-bit half of the four words decides one
    of the eight columns, low halves first."""
    seed, offset = rng[0], rng[1]
    g, m = torch.arange(n // 8, device=rng.device), torch.arange(M, device=rng.device)
    c0, c1 = g[None, :].expand(M, -1), m[:, None].expand(-1, n // 8)
    c2, c3 = offset & _M32, (offset >> 32) & _M32
    k0, k1 = seed & _M32, (seed >> 32) & _M32
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57            # 64-bit products, mod 2^64
        c0, c1, c2, c3 = ((b >> 32) & _M32) ^ c1 ^ k0, b & _M32, ((a >> 32) & _M32) ^ c3 ^ k1, a & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    words = torch.stack(torch.broadcast_tensors(c0, c1, c2, c3), -1)
    halves = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(M, n)
    return halves >= _threshold(p)[0]


def _pack(keep):
    M, n = keep.shape
    bit = 1 << torch.arange(8, device=keep.device, dtype=torch.int32)
    return (keep.reshape(M, n // 8, 8).int() * bit).sum(-1).to(torch.uint8)


def _us_plain(s):
    keep = _keep_plain(s["rng"], s["p"], s["M"], s["n_in"])
    return (s["alpha"] / s["r"] / _threshold(s["p"])[1]) * ((s["x"].float() * keep) @ s["A"].float().T)


def run(s):
    if own:
        import bit_nf4_quantized_11_b200 as q
        if s["op"] == "slots":
            return q.token_slots(s["lengths"], s["slots"], s["tokens"])
        if s["op"] == "keep":
            return q.dropout_keep_bits(s["rng"], s["p"], s["M"], s["n_in"])
        w = q.NF4Weight(rows=s["n_out"], cols=s["n_in"], **s["w"])
        if s["op"] == "multi":
            return q.linear_fwd_slots(s["x"], w, s["A"], s["B"], s["scale"], s["ids"])
        if s["op"] == "fwd":
            h, us = q.linear_fwd_dropout_rng(s["x"], w, s["A"], s["B"], s["alpha"], s["rng"], s["p"])
            return dict(h=h, us=us)
        dx, dA, dB = q.linear_bwd_dropout_rng(s["dh"], s["x"], s["us"], w, s["A"], s["B"], s["alpha"], s["rng"],
                                              s["p"])
        return dict(dx=dx, dA=dA, dB=dB)
    if s["op"] == "slots":
        return _slots_plain(s["lengths"], s["slots"], s["tokens"])
    if s["op"] == "keep":
        return _pack(_keep_plain(s["rng"], s["p"], s["M"], s["n_in"]))
    W = _dequant_plain(s["w"])
    x, A, B = s["x"].float(), s["A"].float(), s["B"].float()
    if s["op"] == "multi":
        # every adapter's rank columns, all but the token's own masked out
        mine = s["ids"][:, None] == torch.arange(s["n"], device=x.device)
        u = (x @ A.reshape(-1, s["n_in"]).T).reshape(s["M"], s["n"], s["r"]) * (mine * s["scale"])[:, :, None]
        h = x @ W.T + u.reshape(s["M"], -1) @ B.transpose(1, 2).reshape(-1, s["n_out"])
        return h.bfloat16()
    if s["op"] == "fwd":
        us = _us_plain(s)
        return dict(h=(x @ W.T + us @ B.T).bfloat16(), us=us.bfloat16())
    scale, kept = s["alpha"] / s["r"], _threshold(s["p"])[1]
    dh, keep = s["dh"].float(), _keep_plain(s["rng"], s["p"], s["M"], s["n_in"])
    du = scale * (dh @ B)
    dx = dh @ W + (du @ A) * keep / kept
    return dict(dx=dx.bfloat16(), dA=du.T @ (x * keep) / kept, dB=dh.T @ s["us"].float())


# ------------------------------------------------------- values in 64 bits
def _exact_weight(w):
    """The stored weight: fp32 scale and product, each rounded, then bf16; exact as fp64."""
    lev = _levels().double().to(w["codes"].device)
    b = w["codes"].int()
    val = torch.stack([lev[b & 15], lev[b >> 4]], -1).flatten().reshape(-1, 64)
    block = torch.arange(w["q8"].numel(), device=val.device)
    c = (w["q8"].double() * w["step2"].double()[block // 256]).float().double()
    c = (c + w["mean"].double()).float().double()
    return (val * c[:, None]).float().bfloat16().double().reshape(b.shape[0], -1)


def _exact_keep(rng, p, M, n):
    """The keep mask by numpy's 64-bit unsigned arithmetic."""
    seed, offset = (np.uint64(int(v) & ((1 << 64) - 1)) for v in rng.tolist())
    m32, sh = np.uint64(_M32), np.uint64(32)
    col, row = np.meshgrid(np.arange(n // 8, dtype=np.uint64), np.arange(M, dtype=np.uint64))
    ctr = [col, row, np.full_like(col, offset & m32), np.full_like(col, offset >> sh)]
    key = [seed & m32, seed >> sh]
    for _ in range(7):
        lo, hi = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(hi >> sh) ^ ctr[1] ^ key[0], hi & m32, (lo >> sh) ^ ctr[3] ^ key[1], lo & m32]
        key = [(key[0] + np.uint64(0x9E3779B9)) & m32, (key[1] + np.uint64(0xBB67AE85)) & m32]
    out = np.empty((M, n), dtype=bool)
    for j in range(8):
        out[:, j::8] = ((ctr[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF)) >= np.uint64(_threshold(p)[0])
    return torch.from_numpy(out).to(rng.device)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "slots":
        ids, end = [], 0
        for n, slot in zip(s["lengths"].tolist(), s["slots"].tolist()):
            ids += [slot] * max(0, n)
        return torch.tensor((ids + [-1] * s["tokens"])[:s["tokens"]], dtype=torch.int32, device="cuda")
    if s["op"] == "keep":
        bits = np.packbits(_exact_keep(s["rng"], s["p"], s["M"], s["n_in"]).cpu().numpy(), axis=1, bitorder="little")
        return torch.from_numpy(bits).cuda()
    W, x, A, B = _exact_weight(s["w"]), s["x"].double(), s["A"].double(), s["B"].double()
    if s["op"] == "multi":
        h = x @ W.T
        for a in range(s["n"]):
            rows = (s["ids"] == a).nonzero().flatten()
            h[rows] += float(s["scale"][a]) * ((x[rows] @ A[a].T) @ B[a].T)
        return h
    kept = 1.0 - _threshold(s["p"])[0] / 65536
    xd, scale = x * _exact_keep(s["rng"], s["p"], s["M"], s["n_in"]) / kept, s["alpha"] / s["r"]
    if s["op"] == "fwd":
        us = scale * (xd @ A.T)
        return dict(h=x @ W.T + us @ B.T, us=us)
    dh = s["dh"].double()
    du = scale * (dh @ B)
    keep = _exact_keep(s["rng"], s["p"], s["M"], s["n_in"])
    return dict(dx=dh @ W + torch.where(keep, du @ A, 0.0) / kept, dA=du.T @ xd, dB=dh.T @ s["us"].double())


# ------------------------------------------------------------------- work
def work(case):
    c = dict(case)
    if c["op"] == "slots":
        return dict(bytes=8 * c["requests"] + 4 * c["tokens"], flops=0)
    if c["op"] == "keep":
        return dict(bytes=16 + c["M"] * c["n_in"] / 8, flops=0)
    M, n_in, n_out, r = c["M"], c["n_in"], c["n_out"], c["r"]
    weight = n_in * n_out * (0.5 + 1 / 64 + 4 / 16384)
    if c["op"] == "multi":
        used = c["n"] * (1 - (1 - 1 / c["n"]) ** c["requests"])          # distinct adapters expected
        return dict(bytes=weight + 2 * M * (n_in + n_out) + 4 * M + used * (2 * r * (n_in + n_out) + 4),
                    flops=2 * M * n_in * n_out + 2 * M * r * (n_in + n_out))
    lora = 2 * r * (n_in + n_out)
    if c["op"] == "fwd":
        return dict(bytes=weight + 2 * M * (n_in + n_out + r) + lora, flops=2 * M * n_in * n_out + M * lora)
    # dx, du, dA and dB; x, dh and us read, dx and the fp32 gradients written
    return dict(bytes=weight + 2 * M * (2 * n_in + n_out + r) + 3 * lora,
                flops=2 * M * n_in * n_out + 2 * M * lora)
