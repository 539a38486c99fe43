// bind.cu — entry points of the Python binding: the arguments of a function
// of include/moe.h as one record of 64-bit numbers, in its order. ctypes takes
// 2.4 us to convert 22 arguments one by one and 0.8 us for a record, which is a
// tenth of a small call.
#include "moe.h"

namespace {

template <typename T>
T* ptr(int64_t v) {
  return reinterpret_cast<T*>(static_cast<uintptr_t>(v));
}
// A number that does not fit an int is refused by the function as a negative one.
int num(int64_t v) { return v > 0x7fffffff || v < -0x7fffffff ? -0x7fffffff : static_cast<int>(v); }
moe_dtype type(int64_t v) { return static_cast<moe_dtype>(v == MOE_F32 || v == MOE_BF16 ? v : 255); }

}  // namespace

extern "C" {

moe_status moe_bind_forward_few(const int64_t* a) {
  return moe_forward_few(ptr<void>(a[0]), ptr<void>(a[1]), ptr<float>(a[2]), ptr<void>(a[3]), ptr<void>(a[4]),
                         ptr<void>(a[5]), num(a[6]), num(a[7]), num(a[8]), num(a[9]), num(a[10]), num(a[11]),
                         type(a[12]), ptr<void>(a[13]), ptr<int32_t>(a[14]), ptr<float>(a[15]), ptr<int32_t>(a[16]),
                         ptr<float>(a[17]), ptr<void>(a[18]), static_cast<size_t>(a[19]), ptr<int32_t>(a[20]),
                         ptr<void>(a[21]));
}

moe_status moe_bind_mx_quantize(const int64_t* a) {
  return moe_mx_quantize(ptr<void>(a[0]), ptr<int32_t>(a[1]), num(a[2]), num(a[3]), num(a[4]), type(a[5]),
                         ptr<void>(a[6]), ptr<void>(a[7]), static_cast<size_t>(a[8]), ptr<void>(a[9]));
}

moe_status moe_bind_mx_dequantize(const int64_t* a) {
  return moe_mx_dequantize(ptr<void>(a[0]), ptr<void>(a[1]), static_cast<size_t>(a[2]), ptr<int32_t>(a[3]), num(a[4]),
                           num(a[5]), num(a[6]), type(a[7]), ptr<void>(a[8]), ptr<void>(a[9]));
}

moe_status moe_bind_mx_matmul(const int64_t* a) {
  return moe_mx_matmul(ptr<void>(a[0]), ptr<void>(a[1]), ptr<void>(a[2]), ptr<void>(a[3]), ptr<int32_t>(a[4]),
                       num(a[5]), num(a[6]), num(a[7]), num(a[8]), type(a[9]), ptr<void>(a[10]), ptr<int32_t>(a[11]),
                       ptr<void>(a[12]));
}

// The weights' six pointers stand in the record, behind the gates.
moe_status moe_bind_mx_experts(const int64_t* a) {
  const moe_mx_weights w = {sizeof(moe_mx_weights), ptr<void>(a[3]), ptr<void>(a[4]), ptr<void>(a[5]),
                            ptr<void>(a[6]),        ptr<void>(a[7]), ptr<void>(a[8])};
  return moe_mx_experts(ptr<void>(a[0]), ptr<int32_t>(a[1]), ptr<float>(a[2]), &w, num(a[9]), num(a[10]), num(a[11]),
                        num(a[12]), num(a[13]), type(a[14]), ptr<void>(a[15]), ptr<int32_t>(a[16]), ptr<void>(a[17]),
                        static_cast<size_t>(a[18]), ptr<int32_t>(a[19]), ptr<void>(a[20]));
}

}  // extern "C"
