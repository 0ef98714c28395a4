// For a test on a host without a GPU: tensors that say they are on a device, and a stand-in for torch's device switch that
// records which device is made current and when the stream is asked for.  Python module `device_recorder`:
//   install()                       takes the place of the switch for devices of type CUDA
//   fake(shape, dtype, index)       a tensor over host memory that says it is on device `index`
//   switches()                      the devices made current since the last call, in order
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Dtype.h>

#include <ATen/ops/from_blob.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>

#include <vector>

namespace {

std::vector<long> g_switches;
c10::DeviceIndex g_current = 0;

struct Recorder final : c10::impl::DeviceGuardImplInterface {
  c10::DeviceType type() const override { return c10::DeviceType::CUDA; }
  c10::Device exchangeDevice(c10::Device d) const override {
    const c10::Device was(type(), g_current);
    setDevice(d);
    return was;
  }
  c10::Device getDevice() const override { return c10::Device(type(), g_current); }
  void setDevice(c10::Device d) const override {
    if (d.index() != g_current) g_switches.push_back(d.index());
    g_current = d.index();
  }
  void uncheckedSetDevice(c10::Device d) const noexcept override { setDevice(d); }
  c10::Stream getStream(c10::Device d) const override { return c10::Stream(c10::Stream::DEFAULT, d); }
  c10::Stream exchangeStream(c10::Stream s) const override { return s; }
  c10::DeviceIndex deviceCount() const noexcept override { return 2; }
};

PyObject* install(PyObject*, PyObject*) {
  static Recorder r;
  c10::impl::device_guard_impl_registry[static_cast<size_t>(c10::DeviceType::CUDA)].store(&r);
  Py_RETURN_NONE;
}

PyObject* fake(PyObject*, PyObject* args) {
  PyObject *shape, *dtype;
  int index;
  if (!PyArg_ParseTuple(args, "OOi", &shape, &dtype, &index)) return nullptr;
  std::vector<int64_t> sizes;
  for (Py_ssize_t i = 0; i < PyTuple_Size(shape); ++i) sizes.push_back(PyLong_AsLongLong(PyTuple_GetItem(shape, i)));
  alignas(64) static char memory[1 << 16];
  const c10::Device dev(c10::DeviceType::CUDA, (c10::DeviceIndex)index);
  const auto type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  return THPVariable_Wrap(at::for_blob(memory, sizes).target_device(dev).options(at::TensorOptions().dtype(type).device(dev))
                              .make_tensor());
}

PyObject* switches(PyObject*, PyObject*) {
  PyObject* list = PyList_New(0);
  for (long d : g_switches) {
    PyObject* o = PyLong_FromLong(d);
    PyList_Append(list, o);
    Py_DECREF(o);
  }
  g_switches.clear();
  return list;
}

PyMethodDef methods[] = {{"install", install, METH_NOARGS, nullptr},
                         {"fake", fake, METH_VARARGS, nullptr},
                         {"switches", switches, METH_NOARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "device_recorder", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_device_recorder() { return PyModule_Create(&module); }
