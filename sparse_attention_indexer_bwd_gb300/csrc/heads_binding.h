// The functions of heads_binding.cpp, in the module's table beside those of train_binding.cpp.
#pragma once
#include <Python.h>

PyObject* qk_norm_rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n);
PyObject* cache_attention(PyObject*, PyObject* const* a, Py_ssize_t n);
