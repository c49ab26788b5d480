"""Host-side argument checks of the 4-bit and log-probability entry points, called with addresses that
are never dereferenced.  Every call here must return during host validation; the module is only run in
a child process that sees no GPU.  Run as a script it prints the return codes as JSON."""
import json
import sys

from speculative_decoding_tree_spec_gb300 import binding

FAKE = 1 << 20  # an aligned address that the host never dereferences
NAN, INF = float("nan"), float("inf")
BIG = (1 << 24) + 1

QUANTIZE = [
    (dict(rows=0), 0),
    (dict(rows=0, x=None, codes=None, scales=None), 0),
    (dict(rows=-1), -1),
    (dict(cols=0), -1),
    (dict(pitch=63), -1),
    (dict(dtype=2), -2),
    (dict(format=2), -2),
    (dict(format=-1), -2),
    (dict(scale=2.0), -1),
    (dict(scale=0.0, format=1), -1),
    (dict(scale=-1.0, format=1), -1),
    (dict(scale=0.75, format=1), -1),
    (dict(scale=NAN, format=1), -1),
    (dict(scale=INF, format=1), -1),
    (dict(scale=2.0 ** -101, format=1), -1),
    (dict(scale=2.0 ** 101, format=1), -1),
    (dict(scale=1e-40, format=1), -1),
    (dict(rows=0, scale=2.0 ** -100, format=1), 0),
    (dict(x=None), -1),
    (dict(codes=None), -1),
    (dict(scales=None), -1),
    (dict(x=FAKE + 8), -3),
    (dict(codes=FAKE + 4), -3),
    (dict(scales=FAKE + 1), -3),
    (dict(pitch=66), -3),
    (dict(pitch=68, dtype=1), -3),
    (dict(rows=BIG), -6),
    (dict(cols=BIG, pitch=BIG), -6),
    (dict(rows=1 << 24, cols=1 << 24, pitch=1 << 24), -6),
    (dict(pitch=1 << 61), -6),
]

LINEAR = [
    (dict(R=0), 0),
    (dict(R=-1), -1),
    (dict(V=0), -1),
    (dict(K=0), -1),
    (dict(pitch=63), -1),
    (dict(dtype=2), -2),
    (dict(format=2), -2),
    (dict(alpha=NAN), -1),
    (dict(alpha=INF), -1),
    (dict(alpha=-INF), -1),
    (dict(a=None), -1),
    (dict(a_scales=None), -1),
    (dict(w=None), -1),
    (dict(w_scales=None), -1),
    (dict(out=None), -1),
    (dict(a=FAKE + 8), -3),
    (dict(a_scales=FAKE + 4), -3),
    (dict(w=FAKE + 2), -3),
    (dict(w_scales=FAKE + 1), -3),
    (dict(out=FAKE + 8), -3),
    (dict(pitch=66), -3),
    (dict(pitch=68, dtype=1), -3),
    (dict(R=BIG), -6),
    (dict(V=BIG, pitch=BIG + 7), -6),
    (dict(K=BIG), -6),
    (dict(V=1 << 24, K=1 << 24, pitch=1 << 24), -6),
    (dict(R=1 << 24, V=1 << 24, pitch=1 << 24), -6),
    (dict(pitch=1 << 60), -6),
]

LOGPROBS = [
    (dict(R=0), 0),
    (dict(R=0, rows=None, n=0, logits=None), 0),
    (dict(R=-1), -1),
    (dict(n=-1), -1),
    (dict(V=0), -1),
    (dict(G=-1), -1),
    (dict(k=-1), -1),
    (dict(k=33), -1),
    (dict(k=5, V=4), -1),
    (dict(dtype=2), -2),
    (dict(T=0.0), -1),
    (dict(T=-1.0), -1),
    (dict(T=NAN), -1),
    (dict(T=INF), -1),
    (dict(T=1e-38), -1),
    (dict(rows=None, R=5), -1),
    (dict(pitch=63), -1),
    (dict(logits=None), -1),
    (dict(tokens=None), -1),
    (dict(lp=None), -1),
    (dict(top=None), -1),
    (dict(top_lp=None), -1),
    (dict(logits=FAKE + 8), -3),
    (dict(pitch=66), -3),
    (dict(pitch=68, dtype=1), -3),
    (dict(V=(1 << 21) + 1, pitch=1 << 22), -6),
    (dict(pitch=1 << 61), -6),
]

FUSED = [
    (dict(R=0), 0),
    (dict(format=2), -2),
    (dict(R=-1), -1),
    (dict(V=0), -1),
    (dict(d=0), -1),
    (dict(k=0), -1),
    (dict(k=33), -1),
    (dict(k=5, V=4), -1),
    (dict(T=0.0), -1),
    (dict(T=NAN), -1),
    (dict(feature_scale=0.3, format=1), -1),
    (dict(weight_scale=0.0, format=1), -1),
    (dict(feature_scale=2.0), -1),
    (dict(weight_scale=0.5), -1),
    (dict(feature_scale=2.0 ** 100, weight_scale=2.0 ** 100, format=1), -1),
    (dict(features=None), -1),
    (dict(w=None), -1),
    (dict(w_scales=None), -1),
    (dict(tokens=None), -1),
    (dict(probs=None), -1),
    (dict(ws=None), -1),
    (dict(features=FAKE + 8), -3),
    (dict(w=FAKE + 8), -3),
    (dict(w_scales=FAKE + 4), -3),
    (dict(d=60), -3),
    (dict(logits=FAKE, pitch=63), -1),
    (dict(logits=FAKE, pitch=68), -3),
    (dict(logits=FAKE + 2, pitch=64), -3),
    (dict(ws_bytes=100), -4),
    (dict(ws=FAKE + 16), -4),
    (dict(V=(1 << 21) + 1), -6),
    (dict(R=BIG), -6),
    (dict(d=BIG + 7), -6),
]


def quantize(L, back, x=FAKE, dtype=0, rows=4, cols=64, pitch=64, format=0, scale=1.0, codes=FAKE, scales=FAKE):
    if back:
        return L.spec_fp4_dequantize(codes, scales, rows, cols, format, scale, x, dtype, pitch, None)
    return L.spec_fp4_quantize(x, dtype, rows, cols, pitch, format, scale, codes, scales, None)


def linear(L, a=FAKE, a_scales=FAKE, w=FAKE, w_scales=FAKE, format=0, R=4, V=64, K=64, alpha=1.0, out=FAKE, dtype=0,
           pitch=64):
    return L.spec_fp4_linear(a, a_scales, w, w_scales, format, R, V, K, alpha, out, dtype, pitch, None)


def logprobs(L, logits=FAKE, dtype=0, n=4, V=64, pitch=64, rows=FAKE, R=4, tokens=FAKE, G=1, k=2, T=1.0, lp=FAKE,
             entropy=FAKE, top=FAKE, top_lp=FAKE, status=FAKE):
    return L.spec_token_logprobs(logits, dtype, n, V, pitch, rows, R, tokens, G, k, T, lp, entropy, top, top_lp,
                                 status, None)


def fused(L, features=FAKE, feature_scale=1.0, w=FAKE, w_scales=FAKE, format=0, weight_scale=1.0, d=64, R=4, V=64, k=2,
          T=1.0, logits=None, pitch=0, tokens=FAKE, probs=FAKE, status=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return L.spec_draft_topk_fused_fp4(features, feature_scale, w, w_scales, format, weight_scale, d, R, V, k, T,
                                       logits, pitch, tokens, probs, status, ws, ws_bytes, None)


def main():
    L = binding.lib()
    json.dump({"quantize": [quantize(L, False, **kw) for kw, _ in QUANTIZE],
               "dequantize": [quantize(L, True, **kw) for kw, _ in QUANTIZE],
               "fused": [fused(L, **kw) for kw, _ in FUSED],
               "linear": [linear(L, **kw) for kw, _ in LINEAR],
               "logprobs": [logprobs(L, **kw) for kw, _ in LOGPROBS]}, sys.stdout)


if __name__ == "__main__":
    main()
