"""The layer with one adapter per row, by definition, in fp64.  Test
infrastructure: see ``oracle/__init__``.

One frozen base serves several adapters [P2 "Training setup versus deployment
setup"]; row i of a batch uses adapter a = ids[i], none when the id lies
outside [0, count).  A [count x r x k], B [count x n x r], s [count]:

    Y[i]  = X[i] W^T + T[i] B_a^T,        T[i] = s_a X[i] A_a^T
    dX[i] = dY[i] W^ + U[i] A_a,          U[i] = s_a dY[i] B_a
    dA_a  = sum over a's rows of U[i]^T X[i]
    dB_a  = sum over a's rows of dY[i]^T T[i]

Each adapter's rows go through the one-adapter functions of ``linear``.
"""

import numpy as np

from . import linear


def rows_of(ids, a):
    return np.nonzero(np.asarray(ids) == a)[0]


def lora_t(X, A, s, ids):
    T = np.zeros((X.shape[0], A.shape[1]))
    for a in range(A.shape[0]):
        i = rows_of(ids, a)
        T[i] = linear.lora_t(X[i], A[a], s[a])
    return T


def fwd(X, W_hat, A, B, s, ids):
    Y = linear.fwd(X, W_hat)
    for a in range(A.shape[0]):
        i = rows_of(ids, a)
        Y[i] = linear.fwd(X[i], W_hat, A[a], B[a], s[a])
    return Y


def bwd(dY, X, T, W_hat, A, B, s, ids):
    """(dX, dA, dB); T [m x r] as the forward kept it."""
    dX = linear.bwd_dx(dY, W_hat)
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for a in range(A.shape[0]):
        i = rows_of(ids, a)
        dX[i] = linear.bwd_dx(dY[i], W_hat, A[a], B[a], s[a])
        dA[a] = linear.lora_u(dY[i], B[a], s[a]).T @ np.asarray(X[i], dtype=np.float64)
        dB[a] = np.asarray(dY[i], dtype=np.float64).T @ np.asarray(T[i], dtype=np.float64)
    return dX, dA, dB
