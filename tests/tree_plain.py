"""The attention of drafted trees in 64 bits by torch, for batches that the numpy oracle is slow on."""
from __future__ import annotations

import numpy as np

import oracle.cache_oracle as co


def plain_attn(torch, c, Q, K, V, sees, offsets, scale):
    """(O, LSE, A, E) of tree_oracle.attn: A = sum p |v|, E the row's largest scale sum |q k|.  Hidden keys are not read."""
    val = torch.from_numpy(co.E4M3).cuda()
    T, Hq, d = Q.shape
    Hkv = K.shape[1]
    g = Hq // Hkv
    page = c["k8"].shape[2]
    f64 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda().double()
    O, A = (torch.zeros((T, Hq, d), dtype=torch.float64, device="cuda") for _ in range(2))
    LSE = torch.full((Hq, T), -np.inf, dtype=torch.float64, device="cuda")
    E = torch.zeros((Hq, T), dtype=torch.float64, device="cuda")
    for s, L in enumerate(c["lens"]):
        a, b, L = int(offsets[s]), int(offsets[s + 1]), int(L)
        if a == b:
            continue
        ids = c["table"][s][: -(-L // page)]

        def keys(w, own):  # [Hkv, cached + own, d]
            x = val[torch.from_numpy(c[w + "8"][ids].astype(np.int64)).cuda()] * f64(c[w + "s"][ids])[..., None, None]
            x = x.transpose(0, 1).reshape(Hkv, -1, d)[:, :L]
            return torch.cat([x, f64(own[a:b]).transpose(0, 1)], 1)
        see = torch.cat([torch.ones((b - a, L), dtype=torch.bool, device="cuda"), torch.from_numpy(sees[s]).cuda()], 1)
        used = see.any(0)
        k, v = (torch.where(used[:, None], keys(w, x), 0.0) for w, x in (("k", K), ("v", V)))
        k, v = (x.repeat_interleave(g, 0) for x in (k, v))
        q = f64(Q[a:b]).transpose(0, 1)
        z = (q @ k.transpose(1, 2) * scale).masked_fill_(~see, -np.inf)
        lse = torch.logsumexp(z, 2)
        p = torch.exp(z - torch.where(torch.isfinite(lse), lse, 0.0)[..., None])
        O[a:b], A[a:b], LSE[:, a:b] = (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1), lse
        E[:, a:b] = (q.abs() @ k.abs().transpose(1, 2) * scale).masked_fill_(~see, 0.0).amax(2)
    return tuple(x.cpu().numpy() for x in (O, LSE, A, E))
