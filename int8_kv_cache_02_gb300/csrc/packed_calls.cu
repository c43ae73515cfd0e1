// The calls of a decoding step with their arguments as an array of 64-bit words, each word read as the
// type that the call's own declaration has in its place.
#include <cstring>
#include <type_traits>
#include <utility>

#include "internal.h"

namespace {

template <class T>
T word(const int64_t* at) {
  if constexpr (std::is_pointer_v<T>) {
    return reinterpret_cast<T>(static_cast<uintptr_t>(*at));
  } else if constexpr (std::is_floating_point_v<T>) {
    double d;
    std::memcpy(&d, at, sizeof(d));
    return static_cast<T>(d);
  } else {
    return static_cast<T>(*at);
  }
}

// Whether a word is a value of the type: an integer that does not fit would become another one.
template <class T>
bool fits(int64_t x) {
  if constexpr (std::is_integral_v<T>) return static_cast<T>(x) == x;
  return true;
}

template <class... A, size_t... I>
int call(int (*f)(A...), const int64_t* words, std::index_sequence<I...>) {
  if (!(fits<A>(words[I]) && ...)) return INT8KV_ERR_INVALID_ARG;
  return f(word<A>(words + I)...);
}

template <class... A>
int call(int (*f)(A...), const int64_t* words) {
  if (!words) return INT8KV_ERR_NULL_PTR;
  return call(f, words, std::index_sequence_for<A...>());
}

}  // namespace

extern "C" {

int kv_rope_append_packed(const int64_t* words) { return call(kv_rope_append, words); }

int attn_decode_scored_int8_packed(const int64_t* words) {
  return call(attn_decode_scored_int8, words);
}

int attn_prefill_chunk_scored_int8_packed(const int64_t* words) {
  return call(attn_prefill_chunk_scored_int8, words);
}

int kv_verify_drafts_packed(const int64_t* words) { return call(kv_verify_drafts, words); }

}  // extern "C"
