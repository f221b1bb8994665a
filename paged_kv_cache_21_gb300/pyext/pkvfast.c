/*
 * _pkvfast: low-overhead Python entry points for the per-step calls of
 * libpagedkv.so (paged_decode, paged_decode_step, paged_decode_attention,
 * kv_append, paged_tree_attention, kv_tree_verify, kv_tree_compact, kv_append_rotary,
 * kv_latent_append, paged_latent_attention).  Argument marshalling only: each function parses plain Python
 * integers and floats (addresses as integers, the CUDA stream as an
 * integer) and calls the C ABI function of the same name, returning its
 * status.  The ctypes binding marshals the same calls about 10 us slower
 * per call, which bounds a Python loop of small decode steps.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stddef.h>
#include <stdint.h>

#include "paged_kv.h"

#define PTR(x) ((void*)(uintptr_t)(x))

static PyObject* fast_paged_decode(PyObject* self, PyObject* args)
{
    unsigned long long out, q, k_new, v_new, k_cache, v_cache, bt, ctx, chunks, seq_chunk, ws,
        ws_bytes, stream;
    int out_dtype, kv_dtype, num_blocks, max_blocks, num_seqs, hq, hkv, d, num_chunks;
    float k_scale, v_scale, scale;
    unsigned int flags;
    (void)self;
    if (!PyArg_ParseTuple(args, "KiKKKKKiffiKiKiiiifKKiIKKK", &out, &out_dtype, &q, &k_new,
                          &v_new, &k_cache, &v_cache, &kv_dtype, &k_scale, &v_scale,
                          &num_blocks, &bt, &max_blocks, &ctx, &num_seqs, &hq, &hkv, &d, &scale,
                          &chunks, &seq_chunk, &num_chunks, &flags, &ws, &ws_bytes, &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = paged_decode(PTR(out), out_dtype, PTR(q), PTR(k_new), PTR(v_new), PTR(k_cache),
                      PTR(v_cache), kv_dtype, k_scale, v_scale, num_blocks,
                      (const int32_t*)PTR(bt), max_blocks, (const int32_t*)PTR(ctx), num_seqs,
                      hq, hkv, d, scale, (const int32_t*)PTR(chunks),
                      (const int32_t*)PTR(seq_chunk), num_chunks, flags, PTR(ws),
                      (size_t)ws_bytes, PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_paged_decode_step(PyObject* self, PyObject* args)
{
    unsigned long long out, q, k_new, v_new, k_cache, v_cache, bt, ctx, ws, ws_bytes, stream;
    int out_dtype, kv_dtype, num_blocks, max_blocks, num_seqs, hq, hkv, d;
    float k_scale, v_scale, scale;
    (void)self;
    if (!PyArg_ParseTuple(args, "KiKKKKKiffiKiKiiiifKKK", &out, &out_dtype, &q, &k_new, &v_new,
                          &k_cache, &v_cache, &kv_dtype, &k_scale, &v_scale, &num_blocks, &bt,
                          &max_blocks, &ctx, &num_seqs, &hq, &hkv, &d, &scale, &ws, &ws_bytes,
                          &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = paged_decode_step(PTR(out), out_dtype, PTR(q), PTR(k_new), PTR(v_new), PTR(k_cache),
                           PTR(v_cache), kv_dtype, k_scale, v_scale, num_blocks,
                           (const int32_t*)PTR(bt), max_blocks, (const int32_t*)PTR(ctx),
                           num_seqs, hq, hkv, d, scale, PTR(ws), (size_t)ws_bytes, PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_paged_decode_attention(PyObject* self, PyObject* args)
{
    unsigned long long out, q, k_cache, v_cache, bt, ctx, ws, ws_bytes, stream;
    int out_dtype, kv_dtype, num_blocks, max_blocks, num_seqs, hq, hkv, d;
    float k_scale, v_scale, scale;
    (void)self;
    if (!PyArg_ParseTuple(args, "KiKKKiffiKiKiiiifKKK", &out, &out_dtype, &q, &k_cache,
                          &v_cache, &kv_dtype, &k_scale, &v_scale, &num_blocks, &bt,
                          &max_blocks, &ctx, &num_seqs, &hq, &hkv, &d, &scale, &ws, &ws_bytes,
                          &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = paged_decode_attention(PTR(out), out_dtype, PTR(q), PTR(k_cache), PTR(v_cache),
                                kv_dtype, k_scale, v_scale, num_blocks,
                                (const int32_t*)PTR(bt), max_blocks, (const int32_t*)PTR(ctx),
                                num_seqs, hq, hkv, d, scale, PTR(ws), (size_t)ws_bytes,
                                PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_kv_append(PyObject* self, PyObject* args)
{
    unsigned long long k, v, k_cache, v_cache, slots, stream;
    int num_tokens, hkv, d, num_blocks, kv_dtype;
    float k_scale, v_scale;
    (void)self;
    if (!PyArg_ParseTuple(args, "KKKKKiiiiiffK", &k, &v, &k_cache, &v_cache, &slots,
                          &num_tokens, &hkv, &d, &num_blocks, &kv_dtype, &k_scale, &v_scale,
                          &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = kv_append(PTR(k), PTR(v), PTR(k_cache), PTR(v_cache), (const int64_t*)PTR(slots),
                   num_tokens, hkv, d, num_blocks, kv_dtype, k_scale, v_scale, PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_paged_tree_attention(PyObject* self, PyObject* args)
{
    unsigned long long out, q, k_cache, v_cache, bt, ctx, starts, parents, ws, ws_bytes, stream;
    int out_dtype, kv_dtype, num_blocks, max_blocks, num_seqs, total, max_nodes, hq, hkv, d;
    float k_scale, v_scale, scale;
    (void)self;
    if (!PyArg_ParseTuple(args, "KiKKKiffiKiKKKiiiiiifKKK", &out, &out_dtype, &q, &k_cache,
                          &v_cache, &kv_dtype, &k_scale, &v_scale, &num_blocks, &bt,
                          &max_blocks, &ctx, &starts, &parents, &num_seqs, &total, &max_nodes,
                          &hq, &hkv, &d, &scale, &ws, &ws_bytes, &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = paged_tree_attention(PTR(out), out_dtype, PTR(q), PTR(k_cache), PTR(v_cache), kv_dtype,
                              k_scale, v_scale, num_blocks, (const int32_t*)PTR(bt), max_blocks,
                              (const int32_t*)PTR(ctx), (const int32_t*)PTR(starts),
                              (const int32_t*)PTR(parents), num_seqs, total, max_nodes, hq, hkv,
                              d, scale, PTR(ws), (size_t)ws_bytes, PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_kv_tree_verify(PyObject* self, PyObject* args)
{
    unsigned long long lens, nodes, out, target, draft, tokens, parents, starts, au, su, stream;
    long long tstride, dstride;
    int dtype, num_seqs, total, max_nodes, vocab;
    unsigned int flags;
    (void)self;
    if (!PyArg_ParseTuple(args, "KKKKLKLiKKKKKiiiiIK", &lens, &nodes, &out, &target, &tstride,
                          &draft, &dstride, &dtype, &tokens, &parents, &starts, &au, &su,
                          &num_seqs, &total, &max_nodes, &vocab, &flags, &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = kv_tree_verify((int32_t*)PTR(lens), (int32_t*)PTR(nodes), (int32_t*)PTR(out),
                        PTR(target), tstride, PTR(draft), dstride, dtype,
                        (const int32_t*)PTR(tokens), (const int32_t*)PTR(parents),
                        (const int32_t*)PTR(starts), (const float*)PTR(au),
                        (const float*)PTR(su), num_seqs, total, max_nodes, vocab, flags,
                        PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_kv_tree_compact(PyObject* self, PyObject* args)
{
    unsigned long long kc, vc, bt, ctx, starts, nodes, lens, stream;
    int layers, max_blocks, num_seqs, max_nodes, hkv, d, num_blocks, kv_dtype;
    (void)self;
    if (!PyArg_ParseTuple(args, "KKiKiKKKKiiiiiiK", &kc, &vc, &layers, &bt, &max_blocks, &ctx,
                          &starts, &nodes, &lens, &num_seqs, &max_nodes, &hkv, &d, &num_blocks,
                          &kv_dtype, &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = kv_tree_compact((void* const*)PTR(kc), (void* const*)PTR(vc), layers,
                         (const int32_t*)PTR(bt), max_blocks, (const int32_t*)PTR(ctx),
                         (const int32_t*)PTR(starts), (const int32_t*)PTR(nodes),
                         (const int32_t*)PTR(lens), num_seqs, max_nodes, hkv, d, num_blocks,
                         kv_dtype, PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_kv_append_rotary(PyObject* self, PyObject* args)
{
    unsigned long long q_out, q, k, v, kc, vc, slots, positions, freq, stream;
    long long so, sq, sk, sv;
    int rot, num_tokens, hq, hkv, d, num_blocks, kv_dtype;
    unsigned int flags;
    float magnitude, k_scale, v_scale;
    (void)self;
    if (!PyArg_ParseTuple(args, "KLKLKLKLKKKKKiIfiiiiiiffK", &q_out, &so, &q, &sq, &k, &sk, &v, &sv,
                          &kc, &vc, &slots, &positions, &freq, &rot, &flags, &magnitude,
                          &num_tokens, &hq, &hkv, &d, &num_blocks, &kv_dtype, &k_scale, &v_scale,
                          &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = kv_append_rotary(PTR(q_out), so, PTR(q), sq, PTR(k), sk, PTR(v), sv, PTR(kc), PTR(vc),
                          (const int64_t*)PTR(slots), (const int64_t*)PTR(positions),
                          (const float*)PTR(freq), rot, flags, magnitude, num_tokens, hq, hkv, d,
                          num_blocks, kv_dtype, k_scale, v_scale, PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_kv_latent_append(PyObject* self, PyObject* args)
{
    unsigned long long q_out, q, latent, k_rope, weight, cache, slots, positions, freq, stream;
    long long ot, oh, qt, qh, sl, sr;
    int num_tokens, h, l, r, num_blocks;
    unsigned int flags;
    float eps, magnitude;
    (void)self;
    if (!PyArg_ParseTuple(args, "KLLKLLKLKLKfKKKKIfiiiiiK", &q_out, &ot, &oh, &q, &qt, &qh, &latent,
                          &sl, &k_rope, &sr, &weight, &eps, &cache, &slots, &positions, &freq,
                          &flags, &magnitude, &num_tokens, &h, &l, &r, &num_blocks, &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = kv_latent_append(PTR(q_out), ot, oh, PTR(q), qt, qh, PTR(latent), sl, PTR(k_rope), sr,
                          PTR(weight), eps, PTR(cache), (const int64_t*)PTR(slots),
                          (const int64_t*)PTR(positions), (const float*)PTR(freq), flags, magnitude,
                          num_tokens, h, l, r, num_blocks, PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* fast_paged_latent_attention(PyObject* self, PyObject* args)
{
    unsigned long long out, q, cache, bt, ctx, starts, parents, ws, ws_bytes, stream;
    int num_blocks, max_blocks, num_seqs, total, max_nodes, h, l, r;
    float scale;
    (void)self;
    if (!PyArg_ParseTuple(args, "KKKiKiKKKiiiiiifKKK", &out, &q, &cache, &num_blocks, &bt,
                          &max_blocks, &ctx, &starts, &parents, &num_seqs, &total, &max_nodes, &h,
                          &l, &r, &scale, &ws, &ws_bytes, &stream))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = paged_latent_attention(PTR(out), PTR(q), PTR(cache), num_blocks, (const int32_t*)PTR(bt),
                                max_blocks, (const int32_t*)PTR(ctx), (const int32_t*)PTR(starts),
                                (const int32_t*)PTR(parents), num_seqs, total, max_nodes, h, l, r,
                                scale, PTR(ws), (size_t)ws_bytes, PTR(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyMethodDef methods[] = {
    {"paged_decode", fast_paged_decode, METH_VARARGS, "paged_decode of libpagedkv (26 args)"},
    {"paged_decode_step", fast_paged_decode_step, METH_VARARGS,
     "paged_decode_step of libpagedkv (22 args)"},
    {"paged_decode_attention", fast_paged_decode_attention, METH_VARARGS,
     "paged_decode_attention of libpagedkv (20 args)"},
    {"kv_append", fast_kv_append, METH_VARARGS, "kv_append of libpagedkv (13 args)"},
    {"paged_tree_attention", fast_paged_tree_attention, METH_VARARGS,
     "paged_tree_attention of libpagedkv (24 args)"},
    {"kv_tree_verify", fast_kv_tree_verify, METH_VARARGS, "kv_tree_verify of libpagedkv (19 args)"},
    {"kv_tree_compact", fast_kv_tree_compact, METH_VARARGS,
     "kv_tree_compact of libpagedkv (16 args)"},
    {"kv_append_rotary", fast_kv_append_rotary, METH_VARARGS,
     "kv_append_rotary of libpagedkv (25 args)"},
    {"kv_latent_append", fast_kv_latent_append, METH_VARARGS,
     "kv_latent_append of libpagedkv (24 args)"},
    {"paged_latent_attention", fast_paged_latent_attention, METH_VARARGS,
     "paged_latent_attention of libpagedkv (19 args)"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkvfast",
                                    "Low-overhead entry points of libpagedkv.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pkvfast(void) { return PyModule_Create(&module); }
