// What the C entry points of the library share on the host: the calling
// thread's error and path strings, the environment switches, and the checks
// of matrix extents. Defined in gemm_api.hip.
#pragma once

#include <stdint.h>

#include <string>

namespace dgt {

// Start of a call: clears the thread's error and path and reads the
// environment switches.
void begin_call();
// Record an error; returns code.
int fail(int code, const std::string& msg);
// The path of this call: its text, or a function that writes it when it is
// asked for (formatting costs about as much as the checks of a small call).
void set_path(const std::string& text);
void set_path_writer(void (*write)(std::string&));
// GEMM_LOG=debug: one line to stderr with the call's sizes and its path or
// error.
void log_layer_call(const char* op, int64_t M, int64_t N, int64_t K, int status);
// GEMM_LAYER_TILE: the product kernel that the layer entry points must take,
// or null.
const char* forced_layer_tile();

// Byte extent of a row-major [rows, cols] matrix with leading dimension ld.
unsigned __int128 extent_bytes(int64_t rows, int64_t cols, int64_t ld, int elem);
bool overlaps(const void* p, unsigned __int128 np, const void* q, unsigned __int128 nq);

}  // namespace dgt
