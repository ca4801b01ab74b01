"""Caches for the tests of the paged key-value cache (not a test module)."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def numpy_cache(rng, B, Hkv, page, d, dv, lens, spare=4, M=None, unit=False):
    """A cache whose sequences hold pages in random order; spare free pages.
    unit: values are small whole numbers (exact in every type)."""
    lens = np.array(lens, dtype=np.int32)
    held = -(-lens // page)
    M = int(held.max(initial=0)) + 2 if M is None else M
    P = int(held.sum()) + spare
    order = rng.permutation(P)
    table = np.full((B, M), -1, dtype=np.int32)
    ref = np.zeros(P, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    ref[order[:at]] = 1

    def pool(w):
        if unit:
            return rng.integers(-100, 101, size=(P, Hkv, page, w)).astype(np.float32)
        return rng.standard_normal((P, Hkv, page, w)).astype(np.float32)

    return dict(k_pages=pool(d), v_pages=pool(dv), table=table, lens=lens, ref=ref)


def on_gpu(cache, dt):
    """The cache on the device, and its pools as the device has them in 64 bits."""
    dev = {}
    for key, x in cache.items():
        t = torch.tensor(x, device="cuda")
        dev[key] = t.to(DT[dt]) if key.endswith("pages") else t
    host = dict(cache)
    for key in ("k_pages", "v_pages"):
        host[key] = dev[key].double().cpu().numpy()
    return dev, host


def holders(table, lens, page, P):
    """References per page from the sequences alone."""
    ref = np.zeros(P, dtype=np.int64)
    for b in range(table.shape[0]):
        for p in table[b, :-(-int(lens[b]) // page)]:
            ref[p] += 1
    return ref
