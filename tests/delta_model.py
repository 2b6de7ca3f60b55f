"""What the bf16 path of the delta rule with one decay per value head rounds, in 64 bits: one head's sequence in chunks of 64 rows, with its
operands rounded to the values that they are held in, everything else exact."""

import torch

C = 64


def bf16_values(x, n):
    """x as a sum of n bf16 values, the first the nearest, the others of what is left."""
    out = []
    for _ in range(n):
        out.append(x.float().bfloat16().double())
        x = x - out[-1]
    return out


def tf32_values(x):
    """x in fp32 as two values of 11 bits."""
    x = x.float().double()
    out = []
    for _ in range(2):
        m, e = torch.frexp(x)
        out.append(torch.ldexp(torch.round(m * 2048) / 2048, e))
        x = x - out[-1]
    return out


def chunk_matrix(k, g, beta):
    """A of a chunk (k [rows, dk], g, beta [rows]): beta_i exp(G_i - G_j) k_i.k_j below the diagonal."""
    G = g.cumsum(0)
    return torch.tril(beta[:, None] * torch.exp(torch.tril(G[:, None] - G[None])) * (k @ k.T), -1)


def growth(k, g, beta):
    """The largest |A| |(I + A)^-1| of a sequence's chunks (2-norms): what an error of A is multiplied by."""
    most = 0.0
    for a in range(0, k.shape[0], C):
        A = chunk_matrix(k[a:a + C], g[a:a + C], beta[a:a + C])
        T = torch.linalg.inv(torch.eye(A.shape[0], dtype=A.dtype) + A)
        most = max(most, float(torch.linalg.matrix_norm(A, 2) * torch.linalg.matrix_norm(T, 2)))
    return most


def inverse(A):
    """(I + A)^-1: blocks of 16, joined twice through X21 = -X22 (A21 X11) with operands of two tf32 values, without the products of both second
    ones."""
    X, one = torch.zeros(C, C, dtype=torch.float64), torch.eye(16, dtype=torch.float64)

    def product(a, b):
        a, b = tf32_values(a), tf32_values(b)
        return a[0] @ b[0] + a[0] @ b[1] + a[1] @ b[0]

    for o in range(0, C, 16):
        s = slice(o, o + 16)
        X[s, s] = torch.linalg.inv(one + A[s, s])
    for size in (16, 32):
        for o in range(0, C, 2 * size):
            first, second = slice(o, o + size), slice(o + size, o + 2 * size)
            X[second, first] = -product(X[second, second], product(A[second, first], X[first, first]))
    return X


def final_state(k, v, g, beta, S):
    """k [T, dk], v [T, dv], g, beta [T], S [dk, dv]."""
    for at in range(0, k.shape[0], C):
        m = min(C, k.shape[0] - at)
        K, V = (torch.zeros(C, x.shape[1], dtype=torch.float64) for x in (k, v))
        b, G = torch.zeros(C, dtype=torch.float64), torch.zeros(C, dtype=torch.float64)
        K[:m], V[:m], b[:m], G[:m] = k[at:at + m], v[at:at + m], beta[at:at + m], g[at:at + m]
        N = bf16_values(inverse(chunk_matrix(K, G, b)) - torch.eye(C, dtype=torch.float64), 3)
        G = G.cumsum(0)
        R = b[:, None] * V - (b * torch.exp(G))[:, None] * (K @ sum(bf16_values(S, 2)))
        first, second = bf16_values(R, 2)
        U = R + sum(n @ first for n in N) + sum(n @ second for n in N[:2])
        S = torch.exp(G[-1]) * S + (torch.exp(G[-1] - G)[:, None] * K).T @ U
    return S
