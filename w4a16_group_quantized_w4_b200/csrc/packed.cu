// w4_packed: the entry points of the decode step with their arguments in one block of 64-bit words.
#include <cstdint>
#include <cstring>
#include <limits>
#include <tuple>
#include <utility>

#include "../../include/w4a16.h"

namespace {

// One word as a parameter of type T; ok turns false where it does not fit.
template <typename T>
T take(uint64_t word, bool& ok) {
  if constexpr (std::is_pointer<T>::value) {
    return reinterpret_cast<T>(static_cast<uintptr_t>(word));
  } else if constexpr (std::is_floating_point<T>::value) {
    double d;
    std::memcpy(&d, &word, sizeof(d));
    return static_cast<T>(d);
  } else {
    const int64_t v = static_cast<int64_t>(word);
    if (sizeof(T) < 8 && (v < static_cast<int64_t>(std::numeric_limits<T>::min()) ||
                          v > static_cast<int64_t>(std::numeric_limits<T>::max())))
      ok = false;
    return static_cast<T>(v);
  }
}

template <typename... P, size_t... I>
w4_status call(w4_status (*fn)(P...), const uint64_t* words, std::index_sequence<I...>) {
  bool ok = true;
  const std::tuple<P...> args{take<P>(words[I], ok)...};
  return ok ? fn(std::get<I>(args)...) : W4_ERR_INVALID_ARG;
}

template <typename... P>
w4_status unpack(w4_status (*fn)(P...), const uint64_t* block) {
  if (block[0] != sizeof...(P)) return W4_ERR_INVALID_ARG;
  return call(fn, block + 1, std::index_sequence_for<P...>{});
}

}  // namespace

extern "C" w4_status w4_packed(int32_t entry, const void* args) {
  if (!args) return W4_ERR_INVALID_ARG;
  const uint64_t* block = static_cast<const uint64_t*>(args);
  switch (entry) {
    case W4_ENTRY_RMS_ADD: return unpack(w4_rms_add, block);
    case W4_ENTRY_RMS_ADD_Q8: return unpack(w4_rms_add_q8, block);
    case W4_ENTRY_LINEAR_8: return unpack(w4a8_linear, block);
    case W4_ENTRY_KV_WRITE: return unpack(kv_cache_write, block);
    case W4_ENTRY_KV_READ: return unpack(kv_cache_read, block);
    case W4_ENTRY_KV_ATTEND: return unpack(kv_cache_attend, block);
    case W4_ENTRY_LINEAR_8S: return unpack(w4a8_linear_s, block);
    default: return W4_ERR_INVALID_ARG;
  }
}
