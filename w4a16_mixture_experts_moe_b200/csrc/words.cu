// The calls of the BF16 products with their arguments as an array of 64-bit
// words: a binding that converts each argument on its own spends more time on
// that than a small call takes on the GPU.
#include <type_traits>

#include "common.cuh"

namespace moe {

// The word as an argument of type T; *fits turns false if T cannot hold it.
template <class T>
static T from_word(int64_t v, bool *fits) {
  if constexpr (std::is_pointer_v<T>) {
    return reinterpret_cast<T>(static_cast<uintptr_t>(v));
  } else {
    *fits &= static_cast<int64_t>(static_cast<T>(v)) == v && (std::is_signed_v<T> || v >= 0);
    return static_cast<T>(v);
  }
}

template <class... A, size_t... I>
static int call_words(const char *who, int (*f)(A...), const int64_t *words, std::index_sequence<I...>) {
  if (!words) return set_error(MOE_ERR_INVALID_ARG, "%s: NULL pointer", who);
  bool fits = true;
  (from_word<A>(words[I], &fits), ...);
  if (!fits) return set_error(MOE_ERR_SHAPE, "%s: a size or flag beyond 32 bits, or a negative number of bytes", who);
  return f(from_word<A>(words[I], &fits)...);
}
template <size_t WORDS, class... A>
static int call_words(const char *who, int (*f)(A...), const int64_t *words) {
  static_assert(sizeof...(A) == WORDS, "the header names the number of words");
  return call_words(who, f, words, std::index_sequence_for<A...>{});
}

}  // namespace moe

extern "C" int moe_grouped_gemm_words(const int64_t *words) {
  return moe::call_words<15>("moe_grouped_gemm", moe_grouped_gemm, words);
}
extern "C" int moe_grouped_gemm_dgrad_words(const int64_t *words) {
  return moe::call_words<15>("moe_grouped_gemm_dgrad", moe_grouped_gemm_dgrad, words);
}
extern "C" int moe_grouped_gemm_wgrad_words(const int64_t *words) {
  return moe::call_words<15>("moe_grouped_gemm_wgrad", moe_grouped_gemm_wgrad, words);
}
extern "C" int moe_lora_linear_words(const int64_t *words) {
  return moe::call_words<20>("moe_lora_linear", moe_lora_linear, words);
}
extern "C" int moe_lora_linear_backward_words(const int64_t *words) {
  return moe::call_words<25>("moe_lora_linear_backward", moe_lora_linear_backward, words);
}
