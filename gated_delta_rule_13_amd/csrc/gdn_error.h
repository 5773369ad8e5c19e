// gdn_error.h -- the calling thread's last error text, shared by the files
// that hold C entry points.
#pragma once
#include <string>

#include "gdn.h"

namespace gdn {
void clear_error();
// Sets the text and returns st.
gdn_status set_error(gdn_status st, const std::string& msg);
// GDN_OK, or GDN_ERR_HIP with the text of the last launch's error.
gdn_status launch_status();
}  // namespace gdn
