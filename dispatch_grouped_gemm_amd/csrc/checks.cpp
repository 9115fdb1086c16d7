// The binding's check of one tensor, in C++: for calls of a few microseconds
// the same comparisons through Python attributes cost more than the launch
// (0.7 us a tensor; here 0.1).
//
//   address(tensor, shape, dtype, device index)
//     the data pointer of a contiguous GPU tensor of that shape, type and
//     device, or -1: the caller then finds out why, and says it.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

// The torch and the Python that this was built for; the binding looks for it in
// the file before it loads it (for others it compares through Python).
extern "C" __attribute__((used)) const char moe_checks_mark[] = CHECKS_MARK;

namespace {

bool as_wanted(PyObject *tensor, PyObject *shape, PyObject *dtype, PyObject *index, void **p)
{
    if (!THPVariable_Check(tensor) || !PyTuple_Check(shape) || !THPDtype_Check(dtype))
        return false;
    const at::Tensor &t = THPVariable_Unpack(tensor);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() ||
        t.scalar_type() != reinterpret_cast<THPDtype *>(dtype)->scalar_type ||
        t.device().index() != PyLong_AsLong(index) || t.dim() != PyTuple_GET_SIZE(shape))
        return false;
    for (int64_t i = 0; i < t.dim(); ++i)
        if (t.size(i) != PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)))
            return false;
    if (!t.is_contiguous())
        return false;
    *p = t.data_ptr();
    return true;
}

PyObject *address(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    void *p = nullptr;
    bool ok = false;
    if (n == 4) {
        try {
            ok = as_wanted(args[0], args[1], args[2], args[3], &p);
        } catch (...) {
            // (a tensor without storage: the caller's own look raises what it has to)
        }
    }
    PyErr_Clear(); // of sizes that are no integers
    return ok ? PyLong_FromVoidPtr(p) : PyLong_FromLong(-1);
}

PyMethodDef methods[] = {
    {"address", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(address)),
     METH_FASTCALL, "Data pointer of a tensor as wanted, or -1."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_checks", nullptr, -1, methods};

} // namespace

PyMODINIT_FUNC PyInit__checks() { return PyModule_Create(&module); }
