// ts_host.hpp -- host helpers shared by the sources of libtopselect.so.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace tsh {

// Records a thread-local message (printf-style) for ts_last_error() and returns `code`.
int fail(int code, const char* fmt, ...);
// TS_OK with the current device in *dev_out if it is a gfx950, else TS_ERR_UNSUPPORTED.
int check_device(int* dev_out);
const char* last_error();
// Workspace bytes of ts_token_logp and ts_cache_evict; 0 for invalid sizes.
size_t token_logp_workspace(int64_t rows, int64_t vocab, int n_top);
size_t cache_evict_workspace(int64_t rows, int64_t slots, int64_t keep_max);

}  // namespace tsh
