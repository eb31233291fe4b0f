// The calling thread's last error message (opt8_last_error), for the host
// files other than opt8_host.cpp, which owns it.
#pragma once

namespace opt8 {

void clear_last_error();
int set_last_error(int code, const char* message);   // returns code

}  // namespace opt8
