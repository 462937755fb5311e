// bind_longctx.hpp -- functions of bind_longctx.cpp that the module's table lists.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

namespace ssm_bind {

PyObject *prefix_attn_fwd(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *page_bounds(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *page_select(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *select_attn_fwd(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *mass_update(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n);

}  // namespace ssm_bind
