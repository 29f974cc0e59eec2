"""fp64 definitions of the operators at the ends of a model.  TEST INFRASTRUCTURE ONLY."""
import numpy as np


def layer_norm(x, weight, bias, eps):
    """(y, xhat, rstd, mean), all fp64; weight and bias may be None."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1, keepdims=True)
    c = x - mean
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
    xhat = c * rstd
    y = xhat if weight is None else xhat * weight
    return (y if bias is None else y + bias), xhat, rstd, mean


def layer_norm_grads(x, weight, eps, dy):
    """(dx, dweight, dbias), fp64."""
    _, xhat, rstd, _ = layer_norm(x, None, None, eps)
    d = dy if weight is None else dy * weight
    dx = rstd * (d - d.mean(axis=1, keepdims=True) - xhat * (d * xhat).mean(axis=1, keepdims=True))
    return dx, (dy * xhat).sum(axis=0), dy.sum(axis=0)


def embedding(ids, weight, scale, ignore_index=-100):
    ids = np.asarray(ids, dtype=np.int64)
    known = (ids != ignore_index) & (ids >= 0) & (ids < len(weight))
    out = np.zeros((len(ids), weight.shape[1]))
    out[known] = scale * weight[ids[known]]
    return out


def embedding_grad(ids, vocab, grad, scale, ignore_index=-100):
    """(gradient (V, H), its absolute terms, tokens of each row)."""
    ids = np.asarray(ids, dtype=np.int64)
    known = (ids != ignore_index) & (ids >= 0) & (ids < vocab)
    out, terms, count = np.zeros((vocab, grad.shape[1])), np.zeros((vocab, grad.shape[1])), np.zeros(vocab)
    np.add.at(out, ids[known], scale * grad[known])
    np.add.at(terms, ids[known], abs(scale) * np.abs(grad[known]))
    np.add.at(count, ids[known], 1)
    return out, terms, count
