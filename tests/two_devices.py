"""Run as a program with a library path, a device order ("1", "01", "threads") and no GPU: every call of the library
linked with tests/fake_cudart.cpp, on each device in turn; prints what device 1 launched, call by call."""
import ctypes
import json
import sys
import threading

from fp4_compressed_sparse_02_gb300 import _lib

P, Q = 0x10000, 0x20000                    # aligned addresses that nothing reads


def args(cls, **kw):
    a = cls()
    a.struct_size = ctypes.sizeof(a)
    for k, v in kw.items():
        part, _, field = k.partition("__")
        setattr(getattr(a, part), field, v) if field else setattr(a, part, v)
    return a


def plane(d, d_ik, fp8=False):
    k = dict(cache__idx_k8=P, cache__idx_k8_scale=P, cache__idx_k_dtype=2) if fp8 else dict(cache__idx_k=P)
    return dict(cache__codes=P, cache__scales=P, cache__page_table=P, cache__num_pages=4096, cache__page_size=64,
                cache__num_seqs=300, cache__max_pages=4096, cache__d=d, cache__d_ik=d_ik, **k)


def norm(T, D, form, unaligned=0, **kw):
    return ("csa2_rms_norm", args(_lib.RmsNormArgs, T=T, D=D, x=P, x_stride=D + unaligned, eps=1e-6, out=P, out_stride=D,
                                  out_form=form, out_scale=P, out4__codes=P, out4__scales=P, out4__rows=T, out4__cols=D, **kw))


def rope(dtype, interleaved, first=0):
    return ("csa2_rope", args(_lib.RopeArgs, T=5000, H=9, D=128, d_rope=64, rot_first=first, x=P, out=Q, x_stride_t=9 * 128,
                              x_stride_h=128, out_stride_t=9 * 128, out_stride_h=128, pos=P, rope_cos=P, rope_sin=P,
                              rope_max_pos=8, dtype=dtype, interleaved=interleaved))


def quant(x_dtype):
    return ("csa2_fp4_quant", args(_lib.Fp4QuantArgs, x=P, x_stride=4096, x_dtype=x_dtype, out__codes=P, out__scales=P,
                                   out__rows=500, out__cols=4096))


def linear(T, K, N):
    return ("csa2_fp4_linear", args(_lib.Fp4LinearArgs, x__codes=P, x__scales=P, x__rows=T, x__cols=K, w__codes=P, w__scales=P,
                                    w__rows=N, w__cols=K, out=P))


def compress(T, d, d_ik, h_dtype=0, m=1):
    return ("csa2_compress_quant", args(_lib.CompressArgs, T=T, m=m, d_model=512, h_dtype=h_dtype, H=P, W_kv=P, W_z=P, seq=P,
                                        entry=P, W_ik=P, **plane(d, d_ik)))


def full(B, H_i, d_ik, fp8=False, group=1, max_n=100000):
    return ("csa2_index_full", args(_lib.IndexFullArgs, B=B, H_i=H_i, q_idx=P, w=P, seq_of=P, n_vis=P, max_n=max_n, num_blocks=2048,
                                    per_block=8, k=512, relu=1, pool=P, pool_len=P, topk=P, topk_len=P, group=group,
                                    **plane(512, d_ik, fp8)))


def attn(Hq, d):
    return ("csa2_sparse_attn", args(_lib.AttnArgs, B=20, Hq=Hq, q=P, seq_of=P, topk=P, topk_len=P, k=512, swa=P, swa_scale=P,
                                     swa_rows=4096, swa_start=P, swa_len=P, swa_max=128, softmax_scale=0.05, out=P, lse=P,
                                     **plane(d, 128)))


CALLS = [norm(5000, D, f) for D in (256, 5120) for f in (0, 2, 3)] + [
    norm(300, D, f, 1) for D in (256, 8000, 20000) for f in (0, 2, 3)] + [
    rope(dt, i, f) for dt in (0, 1) for i in (0, 1) for f in (0, 1)] + [
    ("csa2_rope_table", args(_lib.RopeTableArgs, positions=100000, d_rope=64, theta=1e4, magnitude=1.0, rope_cos=P, rope_sin=P)),
    quant(0), quant(1)] + [
    linear(*s) for s in ((1, 5120, 4096), (20, 1024, 512), (40, 512, 512), (50, 4096, 2560), (100, 4096, 2560), (192, 8192, 5120),
                         (250, 8192, 5120), (120, 512, 1000), (2000, 5120, 8192), (2000, 5120, 8191))] + [
    compress(4, 512, 128), compress(4, 512, 128, 1), compress(300, 512, 128), compress(300, 512, 64), compress(600, 512, 128, m=2),
    compress(2048, 128, 64), full(4, 8, 128), full(300, 8, 128), full(4, 8, 128, True), full(32, 8, 128, group=32),
    full(32, 16, 128, group=16), full(32, 32, 128, group=8), attn(64, 512), attn(8, 128), attn(32, 512)]


def main():
    path, order = sys.argv[1:]
    _lib.LIB_PATH = path
    L = _lib.lib()
    log = (ctypes.c_int * 8192)()

    def call(dev, fn, a):
        L.fake_set_device(dev)
        if not hasattr(L, fn + "_workspace"):
            status = getattr(L, fn)(ctypes.byref(a), None)
        else:
            need = ctypes.c_size_t(0)
            status = getattr(L, fn + "_workspace")(ctypes.byref(a), ctypes.byref(need))
            if status == 0:
                status = getattr(L, fn)(ctypes.byref(a), ctypes.c_void_p(1 << 20), need.value, None)
        return status, L.csa2_last_error_message().decode()

    def launched():
        return [list(log[8 * i:8 * i + 8]) for i in range(L.fake_launches(log, 1024))]

    out = []
    if order == "threads":
        for fn, a in CALLS:
            states, start = [], threading.Barrier(8)

            def one(dev):
                start.wait()
                states.append(call(dev, fn, a))

            t = [threading.Thread(target=one, args=(i % 2,)) for i in range(8)]
            [x.start() for x in t]
            [x.join() for x in t]
            bad = [s for s in states if s[0]]
            out.append([fn, *(bad[0] if bad else (0, "")), sorted(x for x in launched() if x[0] == 1)])
    else:
        for fn, a in CALLS:
            for dev in map(int, order):
                status, message = call(dev, fn, a)
            out.append([fn, status, message if status else "", [x for x in launched() if x[0] == 1]])
    print(json.dumps(out))


if __name__ == "__main__":
    main()
