"""Shared by the tests of the 4-bit product and of the log probabilities: inputs,
and the definitions in 64 bits (plain torch, nothing of the library)."""
import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"nvfp4": 16, "mxfp4": 32}
INF = float("inf")


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def raw_weight(g, fmt, b, n, k, device="cuda"):
    """Weights of random codes (all 16) and random scales (NVFP4: every positive E4M3 value; MXFP4: 2^-20 .. 2^20)."""
    w = {"codes": torch.randint(0, 256, (b, n, k // 2), dtype=torch.uint8, device=device, generator=g), "tensor_scale": None}
    if fmt == "nvfp4":
        w["scales"] = torch.randint(0, 0x7F, (b, n, k // 16), dtype=torch.uint8, device=device, generator=g)
        w["tensor_scale"] = torch.rand(b, device=device, generator=g) + 0.1
    else:
        w["scales"] = torch.randint(107, 148, (b, n, k // 32), dtype=torch.uint8, device=device, generator=g)
    return w


def w64(w, fmt):
    """float64 values [b, n, k] of a weight record."""
    c = w["codes"].int()
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=c.device)
    v = torch.stack((grid[c & 15], grid[c >> 4]), -1).flatten(-2)
    if fmt == "nvfp4":
        s = w["scales"].view(torch.float8_e4m3fn).double().reshape(v.shape[0], v.shape[1], -1) * w["tensor_scale"].double().reshape(-1, 1, 1)
    else:
        s = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device=c.device)[w["scales"].int()]  # (a device's pow is not exact)
    return v * s.repeat_interleave(BLOCK[fmt], -1)


def check_product(y, x, wt, terms):
    """y against x . wt in float64 (x [b, m, c], wt [b, c, o]).

    Operands are exact, products of two bf16 values are exact in f32, so that only
    the sums round: with P = sum |x w|, each of the c `terms` additions is off by a
    step 2^-23 of its partial sum (<= P) at most.  Over all outputs of random data
    a partial sum is of the size sqrt(sum x^2 w^2), and rounding it once every 32
    products, up or down, gives terms sqrt(c / 64) 2^-23 of that in the Frobenius norm;
    the tensor scale's factor 2^-24.  bf16 results: half a step, 2^-8, more."""
    x, wt = x.double(), wt.contiguous()
    e, p, size = torch.matmul(x, wt), torch.matmul(x.abs(), wt.abs()), torch.matmul(x * x, wt * wt).sum().sqrt()
    c = x.shape[-1]
    err = (y.double() - e).abs()
    tol = (terms * c + 16) * 2.0 ** -23 * p
    fro = (terms * max(c / 64, 1.0) ** 0.5 + 2) * 2.0 ** -23 * size
    if y.dtype == torch.bfloat16:
        tol, fro = tol + 2.0 ** -8 * e.abs(), fro + 2.0 ** -8 * e.norm()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol.clamp(min=1e-300)).max()):.3g} of the tolerance"
    assert float(err.norm()) <= float(fro), f"Frobenius {float(err.norm()):.3g}, {float(fro):.3g} allowed"


def logprobs64(logits, targets, temperature=1.0, top=0):
    """The definition in float64, row by row: dict of logprobs, entropy, ranks, top_ids, top_logprobs, lp, M, Z and R = Z - 1, added up without the largest."""
    T, V = logits.shape
    out = {k: [] for k in ("logprobs", "entropy", "ranks", "top_ids", "top_logprobs", "lp", "M", "Z", "R")}
    for i in range(T):
        l = logits[i].double().cpu()
        t = int(targets[i]) if targets is not None else -1
        left = l > -INF
        M = l.max()
        if bool(left.any()):
            z = (l - M) / temperature
            e = torch.exp(z)
            e[int(l.argmax())] = 0.0
            R = e.sum()
            Z = 1 + R
            lp = z - torch.log1p(R)
            H = -(torch.exp(lp[left]) * lp[left]).sum()
        else:
            Z, R, lp, H = 0.0, -1.0, torch.full_like(l, -INF), 0.0
        given = 0 <= t < V
        order = torch.sort(l, descending=True, stable=True).indices
        best = [int(j) for j in order[:top] if l[j] > -INF]
        out["logprobs"].append(float(lp[t]) if given else 0.0)
        out["ranks"].append(int((l > l[t]).sum() + (l[:t] == l[t]).sum()) if given else -1)
        out["entropy"].append(float(H))
        out["top_ids"].append(best + [-1] * (top - len(best)))
        out["top_logprobs"].append([float(lp[j]) for j in best] + [-INF] * (top - len(best)))
        out["lp"].append(lp)
        out["M"].append(float(M))
        out["Z"].append(float(Z))
        out["R"].append(float(R))
    return out
