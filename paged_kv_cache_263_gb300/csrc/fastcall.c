/* fastcall.c -- direct Python entries of the device calls that are about as short as
 * the conversion of their 8 to 26 arguments by ctypes.  An argument is an integer (an
 * address, a size), a float, or None for a null address; the result is the call's
 * kv_status.  The names are those of the C ABI.
 *
 * ctypes takes about 0.15 us an argument: a fork went from 9.2 to 6.7 us, a copy in a
 * layer's two caches from 7.1 to 5.1, attention over 4 short sequences from 11.8 to 9.1
 * (Grace host; programmatic launches of the first two are part of that). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/pagedkv.h"

static void *address(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }

static int32_t int32(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v < INT32_MIN || v > INT32_MAX) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "argument does not fit in 32 bits");
        return -1;
    }
    return (int32_t)v;
}

static int wrong_count(const char *name, Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
    return 1;
}

/* the interpreter may run other threads while a call waits for room in a stream */
#define CALL(expr)                        \
    do {                                  \
        kv_status st;                     \
        if (PyErr_Occurred()) return NULL; \
        Py_BEGIN_ALLOW_THREADS st = expr; \
        Py_END_ALLOW_THREADS return PyLong_FromLong(st); \
    } while (0)

static PyObject *shared_prefix(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (wrong_count("paged_attention_shared_prefix", n, 26)) return NULL;
    void *const out = address(a[0]), *const q = address(a[1]);
    const int32_t *const cu_q = address(a[2]), *const lens = address(a[3]);
    const int32_t seqs = int32(a[4]), rows = int32(a[5]), max_q = int32(a[6]);
    const int32_t *const cu_groups = address(a[7]), *const prefix = address(a[8]);
    const int32_t groups = int32(a[9]), max_prefix = int32(a[10]), max_tail = int32(a[11]);
    const void *const k = address(a[12]), *const v = address(a[13]);
    const int32_t *const tables = address(a[14]);
    const int32_t width = int32(a[15]), hq = int32(a[16]), hkv = int32(a[17]), blocks = int32(a[18]);
    const float scale = (float)PyFloat_AsDouble(a[19]);
    const kv_dtype dtype = (kv_dtype)int32(a[20]);
    const float *const ks = address(a[21]), *const vs = address(a[22]);
    void *const ws = address(a[23]);
    const size_t bytes = PyLong_AsSize_t(a[24]);
    void *const stream = address(a[25]);
    CALL(paged_attention_shared_prefix(out, q, cu_q, lens, seqs, rows, max_q, cu_groups, prefix, groups, max_prefix,
                                       max_tail, k, v, tables, width, hq, hkv, blocks, scale, dtype, ks, vs, ws, bytes,
                                       stream));
}

static PyObject *shared_prefix_workspace(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (wrong_count("paged_attention_shared_prefix_workspace_size", n, 8)) return NULL;
    int32_t v[8];
    for (int i = 0; i < 8; ++i) v[i] = int32(a[i]);
    if (PyErr_Occurred()) return NULL;
    return PyLong_FromSize_t(paged_attention_shared_prefix_workspace_size(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]));
}

/* caches: a list of addresses */
static PyObject *copy_blocks(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (wrong_count("kv_copy_blocks", n, 7)) return NULL;
    if (!PyList_Check(a[0]) || PyList_GET_SIZE(a[0]) > INT32_MAX) {
        PyErr_SetString(PyExc_TypeError, "kv_copy_blocks takes a list of addresses");
        return NULL;
    }
    const int32_t count = (int32_t)PyList_GET_SIZE(a[0]);
    void *few[128], **const caches = count <= 128 ? few : PyMem_Malloc(count * sizeof(void *));
    if (!caches) return PyErr_NoMemory();
    for (int32_t i = 0; i < count; ++i) caches[i] = address(PyList_GET_ITEM(a[0], i));
    const int64_t bytes = PyLong_AsLongLong(a[1]);
    const int32_t blocks = int32(a[2]);
    const int32_t *const src = address(a[3]), *const dst = address(a[4]);
    const int32_t pairs = int32(a[5]);
    void *const stream = address(a[6]);
    kv_status st = KV_ERR_INVALID;
    const int failed = PyErr_Occurred() != NULL;
    if (!failed) {
        Py_BEGIN_ALLOW_THREADS st = kv_copy_blocks(caches, count, bytes, blocks, src, dst, pairs, stream);
        Py_END_ALLOW_THREADS
    }
    if (caches != few) PyMem_Free(caches);
    return failed ? NULL : PyLong_FromLong(st);
}

static PyObject *fork_tables(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (wrong_count("kv_fork_tables", n, 15)) return NULL;
    const int32_t *const tables = address(a[0]);
    const int32_t width = int32(a[1]);
    const int32_t *const lens = address(a[2]);
    const int32_t num_parents = int32(a[3]);
    const int32_t *const parents = address(a[4]);
    const int32_t children = int32(a[5]), keeps = int32(a[6]);
    const int32_t *const free_ids = address(a[7]);
    const int32_t num_free = int32(a[8]);
    int32_t *const child_tables = address(a[9]), *const child_lens = address(a[10]), *const src = address(a[11]),
            *const dst = address(a[12]), *const taken = address(a[13]);
    void *const stream = address(a[14]);
    CALL(kv_fork_tables(tables, width, lens, num_parents, parents, children, keeps, free_ids, num_free, child_tables,
                        child_lens, src, dst, taken, stream));
}

static PyObject *remap_tables(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (wrong_count("kv_remap_tables", n, 8)) return NULL;
    int32_t *const tables = address(a[0]);
    const int32_t width = int32(a[1]);
    const int32_t *const lens = address(a[2]);
    const int32_t seqs = int32(a[3]);
    const int32_t *const src = address(a[4]), *const dst = address(a[5]);
    const int32_t moves = int32(a[6]);
    void *const stream = address(a[7]);
    CALL(kv_remap_tables(tables, width, lens, seqs, src, dst, moves, stream));
}

static PyMethodDef methods[] = {
    {"paged_attention_shared_prefix", (PyCFunction)(void (*)(void))shared_prefix, METH_FASTCALL, NULL},
    {"paged_attention_shared_prefix_workspace_size", (PyCFunction)(void (*)(void))shared_prefix_workspace, METH_FASTCALL, NULL},
    {"kv_copy_blocks", (PyCFunction)(void (*)(void))copy_blocks, METH_FASTCALL, NULL},
    {"kv_fork_tables", (PyCFunction)(void (*)(void))fork_tables, METH_FASTCALL, NULL},
    {"kv_remap_tables", (PyCFunction)(void (*)(void))remap_tables, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&module); }
