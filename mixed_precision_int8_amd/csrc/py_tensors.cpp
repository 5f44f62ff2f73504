// Whether a list of tensors is where it was: for the Python binding only (called with the interpreter's
// lock held, through ctypes.PyDLL), not part of the C ABI.
//
// A set of gradients keeps addresses, and a tensor may be given other memory or another type at any time.
// To ask each one in Python for its address, count and type takes 0.12 us a tensor; DLPack's exchange table
// (version 1, the type's __dlpack_c_exchange_api__) describes one in a tenth of that.
#include <cstdint>

namespace {

// DLPack 1.x, as its specification lays them out
struct DLDevice {
  int32_t type, id;
};
struct DLDataType {
  uint8_t code, bits;
  uint16_t lanes;
};
struct DLTensor {
  void* data;
  DLDevice device;
  int32_t ndim;
  DLDataType dtype;
  int64_t* shape;
  int64_t* strides;
  uint64_t byte_offset;
};
struct DLExchange {
  uint32_t major, minor;
  void* previous;
  void* allocator;
  void* managed_from_object;
  void* managed_to_object;
  int (*tensor_from_object)(void* object, DLTensor* out);
  void* work_stream;
};

struct Look {
  uint64_t address;
  int64_t count;
  DLDataType dtype;
  DLDevice device;
  bool operator==(const Look& o) const {
    return address == o.address && count == o.count && dtype.code == o.dtype.code && dtype.bits == o.dtype.bits &&
           dtype.lanes == o.dtype.lanes && device.type == o.device.type && device.id == o.device.id;
  }
};
static_assert(sizeof(Look) == 32, "the binding's buffers");

}  // namespace

// 1: all n objects are as `seen` says; 0: one is not (write == 0), or all have been written there (write != 0);
// -1: this table does not describe them (an exception may be set).
extern "C" __attribute__((visibility("default"))) int llmint8_py_tensors(const void* table, void* const* objects, int64_t n,
                                                                         void* seen, int write) {
  const DLExchange* x = static_cast<const DLExchange*>(table);
  if (!x || x->major != 1 || !x->tensor_from_object) return -1;
  Look* all = static_cast<Look*>(seen);
  for (int64_t i = 0; i < n; ++i) {
    DLTensor t{};
    if (x->tensor_from_object(objects[i], &t) != 0) return -1;
    Look now{reinterpret_cast<uint64_t>(t.data) + t.byte_offset, 1, t.dtype, t.device};
    for (int d = 0; d < t.ndim; ++d) now.count *= t.shape[d];
    if (write) all[i] = now;
    else if (!(now == all[i])) return 0;
  }
  return write ? 0 : 1;
}
