"""A Performer layer whose row-wise part runs in 8 bits.

The layer of the multi-layer model ("Sub-Linear Memory: How to Make Performers
SLiM", section 2.2) in the form that trains and serves with the 8-bit
operators: root-mean-square norms, no biases, GeLU feed-forward block.  With
the residual stream carried as a pair (x, r) whose sum is the stream, so that
the next norm does the addition:

    h  = x + r              y  = 8 bits of norm(h) g1
    q, k, v = y Wqkv^T      o  = Att^lin(q, k, v)      (causal, the library's)
    h2 = h + 8bits(o) Wo^T  y2 = 8 bits of norm(h2) g2
    z  = y2 W1^T            a  = 8 bits of GeLU(z)
    the next layer's pair: (h2, a W2^T)

What the forward keeps for the backward is 8-bit rows and two fp32 numbers a
row: h, y, o, h2, y2, z and a, 1 byte for each element (5 d_model + 2 d_ff a
token).  q, k, v are formed again from y, and the attention's prefix sums from
them by the library, so no activation is kept in 16 bits.

The computations are the library's; torch moves heads (rows [B L][heads d] to
and from [B][heads][L][d]) and allocates.
"""
import torch

from . import binding, q8


class Layer8:
    """Weights of one layer, packed, with their transposes for the backward.

    heads * d = d_model.  w: the FAVOR+ projection [d, M] or None (elu+1);
    wqkv [3 d_model, d_model], wo [d_model, d_model], w1 [d_ff, d_model],
    w2 [d_model, d_ff] (bf16 or fp32); g1, g2 fp32 [d_model]."""

    NAMES = ("wqkv", "wo", "w1", "w2")

    def __init__(self, heads, w, wqkv, wo, w1, w2, g1, g2, chunk=128, eps=1e-5):
        self.heads, self.w, self.chunk, self.eps = heads, w, chunk, eps
        self.g1, self.g2 = g1, g2
        self.d = g1.shape[0] // heads
        self.load(wqkv=wqkv, wo=wo, w1=w1, w2=w2)

    def load(self, **weights):
        """Pack new values of the named weights (after an optimizer step)."""
        for name, value in weights.items():
            if name not in self.NAMES:
                raise ValueError("no weight %r" % name)
            packed, transposed = q8.pack_weight(value)
            setattr(self, name, packed)
            setattr(self, name + "_t", transposed)

    def _split(self, qkv, b):
        """[B L][3 heads d] -> q, k, v [B, heads, L, d]."""
        length = qkv.shape[0] // b if b else 0
        parts = qkv.view(b, length, 3, self.heads, self.d).permute(2, 0, 3, 1, 4).contiguous()
        return parts[0], parts[1], parts[2]

    @staticmethod
    def _rows(t):
        """[B, heads, L, d] -> [B L][heads d]."""
        b, h, length, d = t.shape
        return t.transpose(1, 2).reshape(b * length, h * d)

    def forward(self, x, r, b):
        """x, r: bf16 rows [B L][d_model] (r None: nothing to add yet), b = B.

        Returns ((h2, f), kept): the next layer's pair and what backward takes."""
        h, y, rstd, h8 = q8.rms_norm(x, self.g1, res=r, eps=self.eps, checkpoint=True)
        q, k, v = self._split(q8.matmul(y, self.wqkv), b)
        o = q8.quantize(self._rows(binding.slim_attn_fwd(q, k, v, self.w, self.chunk)))
        p = q8.matmul(o, self.wo)
        h2, y2, rstd2, h28 = q8.rms_norm(h, self.g2, res=p, eps=self.eps, checkpoint=True)
        a, z8 = q8.gelu(q8.matmul(y2, self.w1))
        return (h2, q8.matmul(a, self.w2)), (b, h8, y, rstd, o, h28, y2, rstd2, z8, a)

    def backward(self, dh2, df, kept):
        """Gradients of forward's pair -> (gradient of x and of r, {name: gradient})."""
        b, h8, y, rstd, o, h28, y2, rstd2, z8, a = kept
        grads = {"w2": q8.wgrad(df, a)}
        da = q8.matmul(q8.quantize(df), self.w2_t)
        dz, dz8 = q8.gelu_bwd(da, z8, quantized=True)
        grads["w1"] = q8.wgrad(dz, y2)
        dh2, grads["g2"] = q8.rms_norm_bwd(q8.matmul(dz8, self.w1_t), h28, rstd2, self.g2, dres=dh2)
        grads["wo"] = q8.wgrad(dh2, o)
        q, k, v = self._split(q8.matmul(y, self.wqkv), b)
        do = q8.matmul(q8.quantize(dh2), self.wo_t)
        do = do.view(b, q.shape[2], self.heads, self.d).transpose(1, 2).contiguous()
        dq, dk, dv, _ = binding.slim_attn_bwd(q, k, v, self.w, do, self.chunk)
        dqkv = torch.cat([self._rows(t) for t in (dq, dk, dv)], dim=1)
        grads["wqkv"] = q8.wgrad(dqkv, y)
        dh, grads["g1"] = q8.rms_norm_bwd(q8.matmul(q8.quantize(dqkv), self.wqkv_t), h8, rstd, self.g1, dres=dh2)
        return dh, grads

    def prefill(self, x, r, b):
        """forward for serving: the next layer's pair, and the attention's state after the rows."""
        h, y, _, _ = q8.rms_norm(x, self.g1, res=r, eps=self.eps)
        q, k, v = self._split(q8.matmul(y, self.wqkv), b)
        state = binding.slim_attn_state(k, v, self.w, self.chunk)
        return self._finish(h, self._rows(binding.slim_attn_fwd(q, k, v, self.w, self.chunk))), state

    def decode(self, x, r, state):
        """One token for each of B sequences: x, r [B][d_model]; state is advanced in place."""
        h, y, _, _ = q8.rms_norm(x, self.g1, res=r, eps=self.eps)
        qkv = q8.matmul(y, self.wqkv).view(x.shape[0], 3, self.heads, self.d).transpose(0, 1).contiguous()
        out = binding.slim_attn_decode(qkv[0], qkv[1], qkv[2], self.w, state)
        return self._finish(h, out.view(x.shape[0], self.heads * self.d))

    def _finish(self, h, o):
        p = q8.matmul(q8.quantize(o), self.wo)
        h2, y2, _, _ = q8.rms_norm(h, self.g2, res=p, eps=self.eps)
        a, _ = q8.gelu(q8.matmul(y2, self.w1), checkpoint=False)
        return h2, q8.matmul(a, self.w2)
