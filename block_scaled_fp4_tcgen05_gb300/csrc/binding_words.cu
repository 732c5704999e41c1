// binding_words.cu -- the calls with many arguments, taking them as one array of
// 64-bit words, for the Python binding (not part of the C ABI of qfp4.h).
//
// ctypes converts every argument by itself, about 0.08 us each: 1.9 us for the
// router's nineteen, where packing them and converting one takes 0.9.
#include <cstddef>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "qfp4.h"

namespace {

template <typename T>
T from_word(int64_t w)
{
    if constexpr (std::is_pointer_v<T>) return reinterpret_cast<T>(static_cast<uintptr_t>(w));
    else return static_cast<T>(w);
}

template <typename... A, size_t... I>
int unpack(int (*f)(A...), const int64_t *w, std::index_sequence<I...>)
{
    return f(from_word<A>(w[I])...);
}

template <typename... A>
int call(int (*f)(A...), const int64_t *w)
{
    return unpack(f, w, std::index_sequence_for<A...>{});
}

}  // namespace

#define QFP4_WORDS(name) \
    extern "C" int name##_words(const int64_t *w) { return call(name, w); }

QFP4_WORDS(qfp4_fp8_quantize)
QFP4_WORDS(qfp4_fp8_quantize_grouped)
QFP4_WORDS(qfp4_fp8_quantize_weight)
QFP4_WORDS(qfp4_gemm_nt_fp8)
QFP4_WORDS(qfp4_gemm_nt_fp8_grouped)
QFP4_WORDS(qfp4_gemm_nt_fp8_kgrouped)
QFP4_WORDS(qfp4_moe_route)
QFP4_WORDS(qfp4_moe_route_backward)
